// Block-scaled FP8 matrix product: out = bf16(A W^T), with E4M3 activations A
// [M, K] (one UE8M0 scale per row and 128 columns) and E4M3 weights W [N, K]
// (one per 128x128 tile):
//   out[m, n] = sum_j 2^(ea(m, j) + ew(n / 128, j)) sum_{k in block j} A[m, k] W[n, k]
// summed in float32 by the matrix cores, which apply the scales themselves,
// and rounded to bf16 once.
#include "iq_common.h"
#include "layer_common.h"

namespace iqp {
namespace {

constexpr int SLAB = 1024;   // bytes of one wave-wide copy to LDS

constexpr int waitcnt_vm(int n) { return (n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14); }

// Tile kernel: a workgroup computes TN weight rows x TM tokens with WN x WM
// waves, all K blocks. Per 128-deep block both operand tiles and the tokens'
// scale words are copied global -> LDS (8 whole rows of 128 bytes a copy, the
// 16-byte chunks of LDS row r permuted by (r / 2) % 8 so that the operand reads
// meet distinct banks), NST blocks in LDS. The product is computed transposed,
// weight rows as the MFMA's rows; weight row n of a 32-row tile sits in LDS
// row 8 ((n / 4) % 4) + 4 (n / 16) + n % 4 of it, so that a lane's sixteen
// accumulators are sixteen consecutive n of one token: 32 bytes of output.
template <int TN, int TM, int NST>
constexpr int tile_lds_bytes() { return NST * (TN * KB + TM * KB + TM * 4); }

template <int TN, int TM, int WN, int WM, int NST>
__device__ __forceinline__ void gemm_tile(const Fp8GemmArgs& p, uint8_t* lds) {
  constexpr int NW = WN * WM;
  constexpr int AN = TN / 32 / WN, AM = TM / 32 / WM;   // 32x32 tiles of a wave
  constexpr int W_BYTES = TN * KB, A_BYTES = TM * KB, S_BYTES = TM * 4;
  constexpr int WC = W_BYTES / SLAB / NW, AC = A_BYTES / SLAB / NW;
  constexpr int SC = (TM / 64 + NW - 1) / NW;           // scale-word copies of a wave (64 words each)
  constexpr int NCOPY = WC + AC + SC;
  static_assert(WC * NW * SLAB == W_BYTES && AC * NW * SLAB == A_BYTES, "whole slabs");
  uint8_t* const lw = lds;
  uint8_t* const la = lds + NST * W_BYTES;
  uint8_t* const ls = la + NST * A_BYTES;

  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave % WN, wm = wave / WN;
  // one XCD (workgroup id mod 8) walks consecutive tiles, tokens first
  const int mt = (int)((p.M + TM - 1) / TM), nt = (int)((p.N + TN - 1) / TN);
  const int64_t total = (int64_t)mt * nt, per = (total + 7) / 8;
  const int64_t tile = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((int64_t)(blockIdx.x >> 3) >= per || tile >= total) return;
  const int64_t n0 = tile / mt * TN, m0 = tile % mt * TM;
  const int nkb = p.nkb;

  const int64_t wrows = p.N - n0 < TN ? p.N - n0 : TN, arows = p.M - m0 < TM ? p.M - m0 : TM;
  const rsrc_t rw = make_rsrc(p.w + n0 * p.ldw, (uint64_t)wrows * p.ldw);
  const rsrc_t ra = make_rsrc(p.a + m0 * p.lda, (uint64_t)arows * p.lda);
  const int64_t nw = (nkb + 3) / 4;
  const rsrc_t rs = make_rsrc(p.a_scales + m0 * p.as_sm, 4 * (uint64_t)((arows - 1) * p.as_sm + (nw - 1) * p.as_sw + 1));

  // copies: slab i of this wave is LDS rows 8 (wave + NW i) + lane / 8
  uint32_t vw[WC], va[AC], vs[SC];
#pragma unroll
  for (int i = 0; i < WC; ++i) {
    const int r = 8 * (wave + NW * i) + (lane >> 3);
    const int n = (r & ~31) + 4 * ((r >> 3) & 3) + 16 * ((r >> 2) & 1) + (r & 3);
    vw[i] = (uint32_t)(n * (int)p.ldw + 16 * ((lane & 7) ^ ((r >> 1) & 7)));
  }
#pragma unroll
  for (int i = 0; i < AC; ++i) {
    const int r = 8 * (wave + NW * i) + (lane >> 3);
    va[i] = (uint32_t)(r * (int)p.lda + 16 * ((lane & 7) ^ ((r >> 1) & 7)));
  }
#pragma unroll
  for (int i = 0; i < SC; ++i) vs[i] = (uint32_t)(4 * (64 * ((wave + NW * i) % (TM / 64)) + lane) * (int)p.as_sm);

  auto copy = [&](int j) __attribute__((always_inline)) {
    const int st = j % NST;
    const uint32_t u = (uint32_t)(KB * j);
#pragma unroll
    for (int i = 0; i < WC; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(lw + st * W_BYTES + SLAB * (wave + NW * i)), 16, vw[i] + u, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < AC; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(la + st * A_BYTES + SLAB * (wave + NW * i)), 16, va[i] + u, 0, 0, 0);
    const uint32_t us = (uint32_t)(4 * (j >> 2) * (int)p.as_sw);
#pragma unroll
    for (int i = 0; i < SC; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(ls + st * S_BYTES + 256 * ((wave + NW * i) % (TM / 64))), 4, vs[i] + us, 0, 0, 0);
  };

  // the weight scales of the wave's 128-row tile, 4 K blocks a lane
  const int64_t wt = (n0 + AN * 32 * wn) / 128;
  const uint8_t* wsc = p.w_scales + (wt < (p.N + 127) / 128 ? wt : (p.N + 127) / 128 - 1) * p.ld_ws;
  uint32_t wsc_lane = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) wsc_lane |= (uint32_t)wsc[4 * lane + b < nkb ? 4 * lane + b : 0] << (8 * b);

  v16f acc[AN][AM];
#pragma unroll
  for (int i = 0; i < AN; ++i)
#pragma unroll
    for (int j = 0; j < AM; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  __builtin_amdgcn_s_waitcnt(WAITCNT_VM0);
#pragma unroll
  for (int j = 0; j < NST - 1; ++j)
    if (j < nkb) copy(j);
  constexpr int WAIT = waitcnt_vm((NST - 2) * NCOPY);
  const int row = lane & 31, swz = (row >> 1) & 7;
  for (int j = 0; j < nkb; ++j) {
    // block j has landed once only the later blocks' copies may be in flight
    if (NST > 2 && j + NST - 2 < nkb)
      __builtin_amdgcn_s_waitcnt(WAIT);
    else
      __builtin_amdgcn_s_waitcnt(WAITCNT_VM0);
    block_barrier();   // block j landed for every wave, block j - 1 read by every wave
    if (j + NST - 1 < nkb) copy(j + NST - 1);
    const int st = j % NST;
    const int ws = (int)((uint32_t)__builtin_amdgcn_readlane((int)wsc_lane, j >> 2) >> (8 * (j & 3)));
    int as[AM];
#pragma unroll
    for (int t = 0; t < AM; ++t)
      as[t] = (int)(*reinterpret_cast<const uint32_t*>(ls + st * S_BYTES + 4 * (32 * (AM * wm + t) + row)) >> (8 * (j & 3)));
#pragma unroll
    for (int kh = 0; kh < 2; ++kh) {
      const int c0 = 4 * kh + 2 * half;
      v8i fw[AN], fa[AM];
#pragma unroll
      for (int t = 0; t < AN; ++t) {
        const uint8_t* b = lw + st * W_BYTES + KB * (32 * (AN * wn + t) + row);
        fw[t] = make_v8i(*reinterpret_cast<const v4u*>(b + 16 * (c0 ^ swz)), *reinterpret_cast<const v4u*>(b + 16 * ((c0 + 1) ^ swz)));
      }
#pragma unroll
      for (int t = 0; t < AM; ++t) {
        const uint8_t* b = la + st * A_BYTES + KB * (32 * (AM * wm + t) + row);
        fa[t] = make_v8i(*reinterpret_cast<const v4u*>(b + 16 * (c0 ^ swz)), *reinterpret_cast<const v4u*>(b + 16 * ((c0 + 1) ^ swz)));
      }
#pragma unroll
      for (int t = 0; t < AN; ++t)
#pragma unroll
        for (int u = 0; u < AM; ++u)
          acc[t][u] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fw[t], fa[u], acc[t][u], 0, 0, 0, ws, 0, as[u]);
    }
  }

#pragma unroll
  for (int u = 0; u < AM; ++u) {
    const int64_t m = m0 + 32 * (AM * wm + u) + row;
    if (m >= p.M) continue;
#pragma unroll
    for (int t = 0; t < AN; ++t) {
      const int64_t n = n0 + 32 * (AN * wn + t) + 16 * half;
      uint16_t* dst = p.out + m * p.ldo + n;
      uint32_t d[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) d[r] = layer::pack_bf16(acc[t][u][2 * r], acc[t][u][2 * r + 1]);
      if (p.wide_out && n + 16 <= p.N) {
        *reinterpret_cast<v4u*>(dst) = v4u{d[0], d[1], d[2], d[3]};
        *reinterpret_cast<v4u*>(dst + 8) = v4u{d[4], d[5], d[6], d[7]};
      } else {
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (n + r < p.N) dst[r] = (uint16_t)(d[r >> 1] >> (16 * (r & 1)));
      }
    }
  }
}

template <int TN, int TM, int WN, int WM, int NST>
__global__ __launch_bounds__(WN * WM * 64)
void fp8_gemm_tile_kernel(Fp8GemmArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[tile_lds_bytes<TN, TM, NST>()];
  gemm_tile<TN, TM, WN, WM, NST>(p, lds);
}

}  // namespace

hipError_t launch_fp8_gemm(const Fp8GemmArgs& p, hipStream_t stream) {
  const int64_t total = ((p.M + 127) / 128) * ((p.N + 127) / 128);
  const int64_t blocks = (total + 7) / 8 * 8;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL((fp8_gemm_tile_kernel<128, 128, 2, 2, 2>), dim3((unsigned)blocks), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace iqp
