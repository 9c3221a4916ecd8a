// Block-scaled FP8 matrix product: out = bf16(A W^T), with E4M3 activations A
// [M, K] (one UE8M0 scale per row and 128 columns) and E4M3 weights W [N, K]
// (one per 128x128 tile):
//   out[m, n] = sum_j 2^(ea(m, j) + ew(n / 128, j)) sum_{k in block j} A[m, k] W[n, k]
// summed in float32 by the matrix cores, which apply the scales themselves,
// and rounded to bf16 once.
//
// Up to 64 tokens the product is bound by the read of the weights (stream
// kernel): 32x7168x8192 13.2 to 14.5 us, 4.1 to 4.5 TB/s of a large copy's 5.1;
// 1x1536x7168 4.9 us, of which launch and first loads are half. Above (tile
// kernel) by the loop around the matrix cores: a K block takes a workgroup 1.28 to
// 1.48 us for its 0.87 us of MFMAs (256x256 tile: 4632x8192x1536 70 us, 1.65 PFLOP/s;
// 4632x8192x7168 266 us, 2.04, as three rounds of tiles for 2.4; a large product of
// the library reaches 2.66), 0.4 us for 0.11 (128x64: 777x2115x7168 23.3 us, 1.0
// PFLOP/s). LDS takes as long as the MFMAs (0.88 us a 256x256 block at 128 bytes a
// cycle, the copies in and the waves' reads), the copies alone more (1.7 us at
// 2048x8192x7168, the whole 1.9). What did not help that loop: more LDS stages, tiles
// in another order (fewer L2 misses, same time), K blocks in another order for
// each workgroup, workgroups that stay and copy the next tile's first blocks
// before they store (72.7 us for 71).
#include <type_traits>

#include "iq_common.h"
#include "layer_common.h"

namespace iqp {
namespace {

constexpr int SLAB = 1024;   // bytes of one wave-wide copy to LDS

constexpr int waitcnt_vm(int n) { return (n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14); }

// A wave's AN x AM accumulator tiles to bf16 rows: weight rows from n0 on,
// tokens from m0 on, the lane's sixteen values of a tile consecutive. They pass
// through the wave's part of LDS (store_bytes<AN>()), 32 tokens at a time, so
// that a store covers whole stretches of a row: 16 bytes a lane where the
// output's alignment allows it, else 2 bytes a lane, 64 consecutive values.
template <int AN>
constexpr int store_bytes() { return 32 * (64 * AN + 16); }

template <int AN, int AM>
__device__ __forceinline__ void store_tile(const Fp8GemmArgs& p, const v16f (&acc)[AN][AM], int64_t n0, int64_t m0, int lane,
                                           uint8_t* lds) {
  constexpr int PITCH = 64 * AN + 16, LANES = 4 * AN;   // bytes of a token's row; 16-byte pieces of it
  const int row = lane & 31, half = lane >> 5;
  const int rows_n = p.N - n0 < 32 * AN ? (int)(p.N - n0) : 32 * AN;
#pragma unroll
  for (int u = 0; u < AM; ++u) {
    const int64_t m = m0 + 32 * u;
    const int rows_m = p.M - m < 32 ? (int)(p.M - m) : 32;
#pragma unroll
    for (int t = 0; t < AN; ++t) {
      uint32_t d[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) d[r] = layer::pack_bf16(acc[t][u][2 * r], acc[t][u][2 * r + 1]);
      uint8_t* const to = lds + row * PITCH + 64 * t + 32 * half;
      *reinterpret_cast<v4u*>(to) = v4u{d[0], d[1], d[2], d[3]};
      *reinterpret_cast<v4u*>(to + 16) = v4u{d[4], d[5], d[6], d[7]};
    }
    asm volatile("" ::: "memory");   // the wave's own writes, then its own reads: in order
    if (p.wide_out && rows_n == 32 * AN) {
#pragma unroll
      for (int i = 0; i < 32; i += 64 / LANES) {
        const int r = i + lane / LANES, c = lane % LANES;
        const v4u v = *reinterpret_cast<const v4u*>(lds + r * PITCH + 16 * c);
        if (r < rows_m) *reinterpret_cast<v4u*>(p.out + (m + r) * p.ldo + n0 + 8 * c) = v;
      }
    } else {
      for (int r = 0; r < rows_m; ++r)
#pragma unroll
        for (int c = 0; c < 32 * AN; c += 64)
          if (c + lane < rows_n) p.out[(m + r) * p.ldo + n0 + c + lane] = *reinterpret_cast<const uint16_t*>(lds + r * PITCH + 2 * (c + lane));
    }
    asm volatile("" ::: "memory");
  }
}

// Tile kernel: a workgroup of WN x WM waves computes TN weight rows x TM tokens,
// K block by K block through NST LDS stages (a block of both operand tiles and
// the tokens' scale words each). Operands are copied global -> LDS, 8 whole rows
// of 128 bytes a copy, the 16-byte chunks of LDS row r permuted by (r / 2) % 8
// so that the operand reads meet distinct banks; copies past the last block read
// zeros out of bounds, which keeps the wait counts constant. The product is
// computed transposed, weight rows as the MFMA's rows; weight row n of a 32-row
// tile sits in LDS row 8 ((n / 4) % 4) + 4 (n / 16) + n % 4 of it, so that a
// lane's sixteen accumulators are sixteen consecutive n of one token: 32 bytes
// of output.
template <int TN, int TM, int WN, int WM, int NST>
constexpr int tile_lds_bytes() {
  constexpr int ring = NST * (TN * KB + TM * KB + TM * 4), out = WN * WM * store_bytes<TN / 32 / WN>();
  return ring > out ? ring : out;
}

// an offset beyond every buffer here: 256 rows of at most 2^22 bytes, 2^28 scale words
constexpr uint32_t PAST = 0x40000000u;

template <int TN, int TM, int WN, int WM, int NST, bool SPLIT>
__device__ __forceinline__ void gemm_tile(const Fp8GemmArgs& p, uint8_t* lds) {
  constexpr int NW = WN * WM;                           // waves
  constexpr int AN = TN / 32 / WN, AM = TM / 32 / WM;   // 32x32 tiles of a wave
  constexpr int W_BYTES = TN * KB, A_BYTES = TM * KB, S_BYTES = TM * 4;
  constexpr int WC = W_BYTES / SLAB / NW, AC = A_BYTES / SLAB / NW;
  constexpr int SW = TM / 64;                           // scale-word copies (64 words each)
  constexpr int SC = (SW + NW - 1) / NW;                // of a wave (some may be made twice)
  constexpr int NCOPY = WC + AC + SC;
  static_assert(WC * NW * SLAB == W_BYTES && AC * NW * SLAB == A_BYTES, "whole slabs");
  static_assert(AN <= 4 && 4 % AN == 0, "a wave's rows share their weight scales");

  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave % WN, wm = wave / WN;
  uint8_t* const lw = lds;
  uint8_t* const la = lw + NST * W_BYTES;
  uint8_t* const ls = la + NST * A_BYTES;
  // one XCD (workgroup id mod 8) walks consecutive tiles, tokens first; SPLIT:
  // piece z of the K blocks of tile `tile`
  const int mt = (int)((p.M + TM - 1) / TM), nt = (int)((p.N + TN - 1) / TN);
  const int64_t total = (int64_t)mt * nt * (SPLIT ? p.splits : 1), per = (total + 7) / 8;
  const int64_t item = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((int64_t)(blockIdx.x >> 3) >= per || item >= total) return;
  const int64_t tile = SPLIT ? item / p.splits : item;
  const int64_t n0 = tile / mt * TN, m0 = tile % mt * TM;
  // blocks [first, nkb)
  const int z = SPLIT ? (int)(item - tile * p.splits) : 0;
  const int first = SPLIT ? p.nkb * z / p.splits : 0, nkb = SPLIT ? p.nkb * (z + 1) / p.splits : p.nkb;

  const int64_t wrows = p.N - n0 < TN ? p.N - n0 : TN, arows = p.M - m0 < TM ? p.M - m0 : TM;
  const rsrc_t rw = make_rsrc(p.w + n0 * p.ldw, (uint64_t)(wrows - 1) * p.ldw + (uint64_t)KB * p.nkb);
  const rsrc_t ra = make_rsrc(p.a + m0 * p.lda, (uint64_t)(arows - 1) * p.lda + (uint64_t)KB * p.nkb);
  const int64_t nw = (p.nkb + 3) / 4;
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
  for (int i = 0; i < SC; ++i) vs[i] = (uint32_t)(4 * (64 * ((wave + NW * i) % SW) + lane) * (int)p.as_sm);

  // copy c (0 .. NCOPY - 1) of block first + i into stage st
  auto copy = [&](int i, int st, int c) __attribute__((always_inline)) {
    const int j = first + i;
    if (c < WC) {
      const uint32_t u = j < nkb ? (uint32_t)(KB * j) : PAST;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(lw + st * W_BYTES + SLAB * (wave + NW * c)), 16, vw[c] + u, 0, 0, 0);
    } else if (c < WC + AC) {
      const uint32_t u = j < nkb ? (uint32_t)(KB * j) : PAST;
      const int k = c - WC;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(la + st * A_BYTES + SLAB * (wave + NW * k)), 16, va[k] + u, 0, 0, 0);
    } else {
      const uint32_t u = j < nkb ? (uint32_t)(4 * (j >> 2) * (int)p.as_sw) : PAST;
      const int k = c - WC - AC;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(ls + st * S_BYTES + 256 * ((wave + NW * k) % SW)), 4, vs[k] + u, 0, 0, 0);
    }
  };

  // the weight scales of the wave's 128-row tile, 4 K blocks a lane
  const int64_t wt = (n0 + AN * 32 * wn) / 128, wt_last = (p.N + 127) / 128 - 1;
  const uint8_t* wsc = p.w_scales + (wt < wt_last ? wt : wt_last) * p.ld_ws;
  uint8_t wb[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) wb[b] = wsc[4 * lane + b < nkb ? 4 * lane + b : 0];
#pragma unroll
  for (int i = 0; i < NST; ++i)
#pragma unroll
    for (int c = 0; c < NCOPY; ++c) copy(i, i, c);
  __builtin_amdgcn_sched_barrier(0);
  uint32_t wsc_lane = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) wsc_lane |= (uint32_t)wb[b] << (8 * b);

  v16f acc[AN][AM];
#pragma unroll
  for (int i = 0; i < AN; ++i)
#pragma unroll
    for (int j = 0; j < AM; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // Half-steps of 64: while the MFMAs of one run, the operands of the next are
  // read. One barrier a block, between its halves: by then every wave has read
  // all of block i, whose stage is refilled, and block i + 1 has landed (only
  // the NST - 2 blocks after it may be in flight).
  constexpr int WAIT = waitcnt_vm((NST - 2) * NCOPY);
  const int row = lane & 31, swz = (row >> 1) & 7;
  const int count = nkb - first;
  v8i fw[2][AN], fa[2][AM];
  uint32_t as_word[AM];
  auto read_half = [&](int st, auto khc) __attribute__((always_inline)) {
    constexpr int kh = decltype(khc)::value;
    const int c0 = 16 * ((4 * kh + 2 * half) ^ swz), c1 = 16 * ((4 * kh + 2 * half + 1) ^ swz);
#pragma unroll
    for (int t = 0; t < AM; ++t) {
      const uint8_t* b = la + st * A_BYTES + KB * (32 * (AM * wm + t) + row);
      fa[kh][t] = make_v8i(*reinterpret_cast<const v4u*>(b + c0), *reinterpret_cast<const v4u*>(b + c1));
    }
#pragma unroll
    for (int t = 0; t < AN; ++t) {
      const uint8_t* b = lw + st * W_BYTES + KB * (32 * (AN * wn + t) + row);
      fw[kh][t] = make_v8i(*reinterpret_cast<const v4u*>(b + c0), *reinterpret_cast<const v4u*>(b + c1));
    }
  };
  auto read_scales = [&](int st) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < AM; ++t) as_word[t] = *reinterpret_cast<const uint32_t*>(ls + st * S_BYTES + 4 * (32 * (AM * wm + t) + row));
  };
  using H0 = std::integral_constant<int, 0>;
  using H1 = std::integral_constant<int, 1>;
  {
    constexpr int FIRST = waitcnt_vm((NST - 1) * NCOPY);
    __builtin_amdgcn_s_waitcnt(FIRST);
  }
  block_barrier();
  read_scales(0);
  read_half(0, H0{});
  for (int i = 0; i < count; ++i) {
    const int st = i % NST, j = first + i;
    const int ws = (int)((uint32_t)__builtin_amdgcn_readlane((int)wsc_lane, (j >> 2) & 63) >> (8 * (j & 3)));
    int as[AM];
#pragma unroll
    for (int t = 0; t < AM; ++t) as[t] = (int)(as_word[t] >> (8 * (j & 3)));
    read_half(st, H1{});
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < AN; ++t)
#pragma unroll
      for (int u = 0; u < AM; ++u)
        acc[t][u] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fw[0][t], fa[0][u], acc[t][u], 0, 0, 0, ws, 0, as[u]);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(WAITCNT_LGKM0);
    __builtin_amdgcn_s_waitcnt(WAIT);
    block_barrier();
    const int st1 = st + 1 < NST ? st + 1 : 0;
    read_scales(st1);
    read_half(st1, H0{});
    __builtin_amdgcn_sched_barrier(0);
    // the copies one by one between the MFMAs: issued together they would hold
    // the wave until the address unit has taken them all
#pragma unroll
    for (int t = 0; t < AN; ++t)
#pragma unroll
      for (int u = 0; u < AM; ++u) {
        acc[t][u] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fw[1][t], fa[1][u], acc[t][u], 0, 0, 0, ws, 0, as[u]);
#pragma unroll
        for (int c = NCOPY * (t * AM + u) / (AN * AM); c < NCOPY * (t * AM + u + 1) / (AN * AM); ++c) copy(i + NST, st, c);
        __builtin_amdgcn_sched_barrier(0);
      }
  }

  if constexpr (SPLIT) {
    // the sums, in the accumulators' order, for fp8_gemm_join_kernel (copies past the
    // last block may be on their way to LDS: a wave's end waits for them)
    float* const to = p.sums + (tile * p.splits + z) * (TN * TM) + wave * (AN * AM * 1024) + 4 * lane;
#pragma unroll
    for (int t = 0; t < AN; ++t)
#pragma unroll
      for (int u = 0; u < AM; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          *reinterpret_cast<v4f*>(to + ((t * AM + u) * 4 + r) * 256) =
              v4f{acc[t][u][4 * r], acc[t][u][4 * r + 1], acc[t][u][4 * r + 2], acc[t][u][4 * r + 3]};
    return;
  }
  // in the ring's place: every wave has read its operands, and no copy is in flight
  __builtin_amdgcn_s_waitcnt(WAITCNT_VM0);
  __syncthreads();
  store_tile<AN, AM>(p, acc, n0 + 32 * AN * wn, m0 + 32 * AM * wm, lane, lds + wave * store_bytes<AN>());
}

template <int TN, int TM, int WN, int WM, int NST, bool SPLIT>
__global__ __launch_bounds__(WN * WM * 64)
void fp8_gemm_tile_kernel(Fp8GemmArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[tile_lds_bytes<TN, TM, WN, WM, NST>()];
  gemm_tile<TN, TM, WN, WM, NST, SPLIT>(p, lds);
}

// Adds up the pieces of a split tile, in their order, and stores it.
template <int TN, int TM, int WN, int WM>
__device__ __forceinline__ void gemm_join(const Fp8GemmArgs& p, uint8_t* lds) {
  constexpr int AN = TN / 32 / WN, AM = TM / 32 / WM;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int mt = (int)((p.M + TM - 1) / TM);
  const int64_t tile = blockIdx.x, n0 = tile / mt * TN, m0 = tile % mt * TM;
  const float* const from = p.sums + tile * p.splits * (TN * TM) + wave * (AN * AM * 1024) + 4 * lane;
  v16f acc[AN][AM];
#pragma unroll
  for (int t = 0; t < AN; ++t)
#pragma unroll
    for (int u = 0; u < AM; ++u)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[t][u][r] = 0.f;
  for (int z = 0; z < p.splits; ++z)
#pragma unroll
    for (int t = 0; t < AN; ++t)
#pragma unroll
      for (int u = 0; u < AM; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const v4f x = *reinterpret_cast<const v4f*>(from + (int64_t)z * (TN * TM) + ((t * AM + u) * 4 + r) * 256);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[t][u][4 * r + e] += x[e];
        }
  store_tile<AN, AM>(p, acc, n0 + 32 * AN * (wave % WN), m0 + 32 * AM * (wave / WN), lane, lds + wave * store_bytes<AN>());
}

template <int TN, int TM, int WN, int WM>
__global__ __launch_bounds__(WN * WM * 64)
void fp8_gemm_join_kernel(Fp8GemmArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[WN * WM * store_bytes<TN / 32 / WN>()];
  gemm_join<TN, TM, WN, WM>(p, lds);
}

// Stream kernel, for few tokens: the product is then a read of the weights. A
// workgroup owns NT = 16 RT weight rows and all (at most 16 MT) tokens; its
// WAVES waves share out the K blocks (wave w takes blocks w, w + WAVES, ...), so
// that small N still spreads over many CUs and no second launch or workspace
// joins partial sums. Each wave streams its blocks' weight and activation rows
// through NST LDS stages of its own: no barrier in the loop, only the wave's
// wait counts. Copies past the last block read zeros out of bounds, which
// keeps the counts constant. The waves' sums meet in LDS at the end. Workgroups
// start the K blocks at different places: in step, all of them would read the
// same few columns of W at a time, whose rows lie at equal strides and share
// memory channels (16x7168x8192: 15.2 us in step, 13.6 with this).
// 16x16x128 MFMA: weight rows as its rows, tokens as its columns.
template <int RT, int MT, int WAVES, int NST>
constexpr int stream_lds_bytes() {
  constexpr int ring = WAVES * NST * ((16 * RT + 16 * MT) * KB + 256);
  constexpr int sums = WAVES * 16 * MT * (16 * RT + 4) * 4;
  return ring > sums ? ring : sums;
}

template <int RT, int MT, int WAVES, int NST>
__device__ __forceinline__ void gemm_stream(const Fp8GemmArgs& p, uint8_t* lds) {
  constexpr int NT = 16 * RT, TOK = 16 * MT;
  constexpr int STAGE = (NT + TOK) * KB + 256;      // weights, activations, scale words
  constexpr int WC = NT / 8, AC = TOK / 8, NCOPY = WC + AC + 1;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * NT;
  const int64_t m0 = (int64_t)blockIdx.y * TOK;
  const int nkb = p.nkb;
  const int rot = (int)((blockIdx.x >> 3) * 5 % 32) % nkb;   // an XCD's neighbours 5 blocks apart
  const int64_t wrows = p.N - n0 < NT ? p.N - n0 : NT, arows = p.M - m0 < TOK ? p.M - m0 : TOK;
  const rsrc_t rw = make_rsrc(p.w + n0 * p.ldw, (uint64_t)(wrows - 1) * p.ldw + (uint64_t)KB * p.nkb);
  const rsrc_t ra = make_rsrc(p.a + m0 * p.lda, (uint64_t)(arows - 1) * p.lda + (uint64_t)KB * p.nkb);
  const int64_t nw = (nkb + 3) / 4;
  const rsrc_t rs = make_rsrc(p.a_scales + m0 * p.as_sm, 4 * (uint64_t)((arows - 1) * p.as_sm + (nw - 1) * p.as_sw + 1));
  // copy c moves rows 8 c + lane / 8, 16-byte chunk permuted by (row / 2) % 8
  uint32_t vw[WC], va[AC];
#pragma unroll
  for (int c = 0; c < WC; ++c) {
    const int r = 8 * c + (lane >> 3);
    vw[c] = (uint32_t)(r * (int)p.ldw + 16 * ((lane & 7) ^ ((r >> 1) & 7)));
  }
#pragma unroll
  for (int c = 0; c < AC; ++c) {
    const int r = 8 * c + (lane >> 3);
    va[c] = (uint32_t)(r * (int)p.lda + 16 * ((lane & 7) ^ ((r >> 1) & 7)));
  }
  const uint32_t vs = lane < TOK ? (uint32_t)(4 * lane * (int)p.as_sm) : PAST;
  uint8_t* const ring = lds + wave * NST * STAGE;

  // block i of this wave into stage st
  auto copy = [&](int i, int st) __attribute__((always_inline)) {
    const int turn = wave + WAVES * i, j = turn + rot < nkb ? turn + rot : turn + rot - nkb;
    const uint32_t u = turn < nkb ? (uint32_t)(KB * j) : PAST;
    uint8_t* const b = ring + st * STAGE;
#pragma unroll
    for (int c = 0; c < WC; ++c)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(b + SLAB * c), 16, vw[c] + u, 0, 0, 0);
#pragma unroll
    for (int c = 0; c < AC; ++c)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(b + NT * KB + SLAB * c), 16, va[c] + u, 0, 0, 0);
    const uint32_t us = turn < nkb ? (uint32_t)(4 * (j >> 2) * (int)p.as_sw) : PAST;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(b + (NT + TOK) * KB), 4, vs + us, 0, 0, 0);
  };

  const uint8_t* wsc = p.w_scales + n0 / 128 * p.ld_ws;
  uint32_t wsc_lane = 0;
  uint8_t wb[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) wb[b] = wsc[4 * lane + b < nkb ? 4 * lane + b : 0];
#pragma unroll
  for (int st = 0; st < NST; ++st) copy(st, st);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int b = 0; b < 4; ++b) wsc_lane |= (uint32_t)wb[b] << (8 * b);

  v4f acc[RT][MT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[r][t] = v4f{0.f, 0.f, 0.f, 0.f};
  const int count = nkb > wave ? (nkb - wave + WAVES - 1) / WAVES : 0;
  constexpr int WAIT = waitcnt_vm((NST - 1) * NCOPY);
  const int swz = (col >> 1) & 7;
  const int c0 = 16 * ((2 * g) ^ swz), c1 = 16 * ((2 * g + 1) ^ swz);
  int st = 0;
  for (int i = 0; i < count; ++i) {
    __builtin_amdgcn_s_waitcnt(WAIT);
    asm volatile("" ::: "memory");
    const int turn = wave + WAVES * i, j = turn + rot < nkb ? turn + rot : turn + rot - nkb;
    const uint8_t* const b = ring + st * STAGE;
    const int ws = (int)((uint32_t)__builtin_amdgcn_readlane((int)wsc_lane, j >> 2) >> (8 * (j & 3)));
    v8i fw[RT], fa[MT];
    int as[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
      as[t] = (int)(*reinterpret_cast<const uint32_t*>(b + (NT + TOK) * KB + 4 * (16 * t + col)) >> (8 * (j & 3)));
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const uint8_t* x = b + KB * (16 * r + col);
      fw[r] = make_v8i(*reinterpret_cast<const v4u*>(x + c0), *reinterpret_cast<const v4u*>(x + c1));
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const uint8_t* x = b + NT * KB + KB * (16 * t + col);
      fa[t] = make_v8i(*reinterpret_cast<const v4u*>(x + c0), *reinterpret_cast<const v4u*>(x + c1));
    }
    // the stage is read: refill it
    __builtin_amdgcn_s_waitcnt(WAITCNT_LGKM0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    copy(i + NST, st);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < MT; ++t)
        acc[r][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw[r], fa[t], acc[r][t], 0, 0, 0, ws, 0, as[t]);
    st = st + 1 < NST ? st + 1 : 0;
  }

  // the waves' sums, [wave][token][row], in the ring's place
  __builtin_amdgcn_s_waitcnt(WAITCNT_VM0);
  __syncthreads();
  constexpr int PITCH = NT + 4;
  float* const sums = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < MT; ++t)
      *reinterpret_cast<v4f*>(sums + ((int64_t)wave * TOK + 16 * t + col) * PITCH + 16 * r + 4 * g) = acc[r][t];
  __syncthreads();
  for (int i = tid; i < (int)arows * (NT / 2); i += WAVES * 64) {
    const int t = i / (NT / 2), n = 2 * (i % (NT / 2));
    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const float* x = sums + (w * TOK + t) * PITCH + n;
      lo += x[0];
      hi += x[1];
    }
    const uint32_t d = layer::pack_bf16(lo, hi);
    uint16_t* const dst = p.out + (m0 + t) * p.ldo + n0 + n;
    if (p.wide_out && n0 + n + 1 < p.N) {
      *reinterpret_cast<uint32_t*>(dst) = d;
    } else {
      if (n0 + n < p.N) dst[0] = (uint16_t)d;
      if (n0 + n + 1 < p.N) dst[1] = (uint16_t)(d >> 16);
    }
  }
}

template <int RT, int MT, int WAVES, int NST>
__global__ __launch_bounds__(WAVES * 64)
void fp8_gemm_stream_kernel(Fp8GemmArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[stream_lds_bytes<RT, MT, WAVES, NST>()];
  gemm_stream<RT, MT, WAVES, NST>(p, lds);
}

template <int RT, int MT, int WAVES, int NST>
hipError_t launch_stream(const Fp8GemmArgs& p, hipStream_t stream) {
  const int64_t nt = (p.N + 16 * RT - 1) / (16 * RT), mt = (p.M + 16 * MT - 1) / (16 * MT);
  if (nt > 0x7FFFFFFF || mt > 65535) return hipErrorInvalidValue;
  hipLaunchKernelGGL((fp8_gemm_stream_kernel<RT, MT, WAVES, NST>), dim3((unsigned)nt, (unsigned)mt), dim3(WAVES * 64), 0, stream, p);
  return hipGetLastError();
}

template <int TN, int TM, int WN, int WM, int NST>
hipError_t launch_tile(const Fp8GemmArgs& p, hipStream_t stream) {
  const int64_t total = ((p.M + TM - 1) / TM) * ((p.N + TN - 1) / TN);
  const int64_t blocks = (total + 7) / 8 * 8;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL((fp8_gemm_tile_kernel<TN, TM, WN, WM, NST, false>), dim3((unsigned)blocks), dim3(WN * WM * 64), 0, stream, p);
  return hipGetLastError();
}

// the 64x64 tile with its K blocks in p.splits pieces
hipError_t launch_split(const Fp8GemmArgs& p, hipStream_t stream) {
  const int64_t tiles = ((p.M + 63) / 64) * ((p.N + 63) / 64), blocks = (tiles * p.splits + 7) / 8 * 8;
  hipLaunchKernelGGL((fp8_gemm_tile_kernel<64, 64, 2, 2, 4, true>), dim3((unsigned)blocks), dim3(256), 0, stream, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((fp8_gemm_join_kernel<64, 64, 2, 2>), dim3((unsigned)tiles), dim3(256), 0, stream, p);
  return hipGetLastError();
}

// The kernels' time in us on a full MI355X, from the sizes alone. A workgroup's K
// block takes a time of its own that more workgroups do not change until every
// CU has one (the loop's copies, reads and barrier follow one another), and
// each further 256 workgroups add to it. Measured over M 96 .. 4632, N 384 ..
// 8192, K 640 .. 7168; us a block for up to 256 workgroups, for up to 512:
//   64x64 0.32, 0.52;  128x64 0.42, 0.69;  128x128 four stages 0.56, 1.13;
//   128x128 two stages 0.75, 0.9;  256x256 1.3, 2.6 (an area 16 times the first's)
// It ranks tiles and is no forecast: 61 us for 4632x8192x1536, which takes 69 to 76,
// and it has no term for bytes.
double tile_us(int64_t M, int64_t N, int64_t nkb, int TN, int TM, double fixed, double block, double more, int group) {
  const int64_t tiles = ((M + TM - 1) / TM) * ((N + TN - 1) / TN);
  const int64_t rounds = (tiles + 255) / 256;
  const int64_t turns = (rounds + group - 1) / group;      // `group` workgroups share a CU
  return turns * fixed + nkb * (turns * block + (rounds - turns) * more);
}

}  // namespace

// Pieces that the K blocks of a product are split into (1: not split): where
// few 64x64 tiles walk many blocks, as many as still give each a CU of its own,
// down to eight blocks a piece, if that takes at least 16 blocks (5 us) off the
// walk: the second launch and the sums' way through memory take 3.5 to 5.
// Measured, split / not, us: 96x384x7168 10.0 / 18.1, 268x1024x7168 13.4 / 18.1,
// 96x384x3200 8.4 / 9.7; 268x1024x3200 10.4 / 9.9 (not split), 268x2115x7168 17.9 / 19.1.
int fp8_gemm_splits(int64_t M, int64_t N, int64_t K) {
  if (M <= 64) return 1;
  const int64_t tiles = ((M + 63) / 64) * ((N + 63) / 64), nkb = K / 128;
  int64_t z = GEMM_SPLIT_GROUPS / tiles;
  if (z > nkb / 8) z = nkb / 8;
  return z >= 2 && nkb - nkb / z >= 16 ? (int)z : 1;
}

GemmKernel fp8_gemm_kernel(int64_t M, int64_t N, int64_t K, int splits) {
  // Up to 64 tokens the product is a read of the weights (64x1500x7168, us: stream
  // kernel 10.1, 64x64 tiles 19.2; 64x7168x8192 20.3, 26.9; 64x4000x1536 5.5, 6.7); 16 or
  // 32 rows of them a workgroup, by which of the two gives the CUs enough
  // workgroups (32 / 16 rows: 16x7168x8192 13.6 / 15.3, 32x7168x8192 15.6 / 20.0,
  // 64x7168x8192 20.3 / 28.3, 40x8192x1536 6.5 / 8.7; 16x1536x7168 7.2 / 5.6,
  // 32x2000x7168 8.6 / 7.0, 64x4000x1536 6.2 / 5.5). Above, it would read the weights
  // once for every 64 tokens (7168x8192, us, tiles / stream kernel by 64 tokens: 65
  // tokens 22.9 / 27.9, 128 22.7 / 32.3, 256 32.9 / 66.4; 64 in one read 17.0).
  if (M <= 64) {
    const bool wide = N >= 6144;
    if (M <= 16) return wide ? GEMM_STREAM_32x16 : GEMM_STREAM_16x16;
    if (M <= 32) return wide ? GEMM_STREAM_32x32 : GEMM_STREAM_16x32;
    return wide ? GEMM_STREAM_32x64 : GEMM_STREAM_16x64;
  }
  if (splits > 1) return GEMM_SPLIT_64x64;
  const int64_t nkb = K / 128;
  const struct {
    GemmKernel kernel;
    double us;
  } tiles[] = {
      {GEMM_TILE_64x64, tile_us(M, N, nkb, 64, 64, 1.5, 0.31, 0.23, 2)},
      {GEMM_TILE_128x64, tile_us(M, N, nkb, 128, 64, 2.0, 0.41, 0.3, 2)},
      {GEMM_TILE_128x128, tile_us(M, N, nkb, 128, 128, 3.0, 0.54, 0.54, 1)},
      {GEMM_TILE_128x128_TWO, tile_us(M, N, nkb, 128, 128, 3.0, 0.73, 0.18, 2)},
      {GEMM_TILE_256x256, tile_us(M, N, nkb, 256, 256, 5.0, 1.28, 1.28, 1)},
  };
  int best = 0;
  for (int i = 1; i < 5; ++i)
    if (tiles[i].us < tiles[best].us) best = i;
  return tiles[best].kernel;
}

const char* fp8_gemm_kernel_name(GemmKernel kernel) {
  switch (kernel) {
    case GEMM_STREAM_16x16: return "stream 16x16";
    case GEMM_STREAM_32x16: return "stream 32x16";
    case GEMM_STREAM_16x32: return "stream 16x32";
    case GEMM_STREAM_32x32: return "stream 32x32";
    case GEMM_STREAM_16x64: return "stream 16x64";
    case GEMM_STREAM_32x64: return "stream 32x64";
    case GEMM_SPLIT_64x64: return "split 64x64";
    case GEMM_TILE_64x64: return "tile 64x64";
    case GEMM_TILE_128x64: return "tile 128x64";
    case GEMM_TILE_128x128: return "tile 128x128";
    case GEMM_TILE_128x128_TWO: return "tile 128x128, two stages";
    case GEMM_TILE_256x256: return "tile 256x256";
  }
  return "";
}

hipError_t launch_fp8_gemm(const Fp8GemmArgs& p, hipStream_t stream) {
  switch (fp8_gemm_kernel(p.M, p.N, (int64_t)p.nkb * 128, p.splits)) {
    case GEMM_STREAM_16x16: return launch_stream<1, 1, 4, 4>(p, stream);
    case GEMM_STREAM_32x16: return launch_stream<2, 1, 8, 3>(p, stream);
    case GEMM_STREAM_16x32: return launch_stream<1, 2, 4, 3>(p, stream);
    case GEMM_STREAM_32x32: return launch_stream<2, 2, 8, 2>(p, stream);
    case GEMM_STREAM_16x64: return launch_stream<1, 4, 4, 3>(p, stream);
    case GEMM_STREAM_32x64: return launch_stream<2, 4, 4, 3>(p, stream);
    case GEMM_SPLIT_64x64: return launch_split(p, stream);
    case GEMM_TILE_64x64: return launch_tile<64, 64, 2, 2, 4>(p, stream);
    case GEMM_TILE_128x64: return launch_tile<128, 64, 2, 2, 3>(p, stream);
    case GEMM_TILE_128x128: return launch_tile<128, 128, 2, 2, 4>(p, stream);
    case GEMM_TILE_128x128_TWO: return launch_tile<128, 128, 2, 2, 2>(p, stream);
    case GEMM_TILE_256x256: return launch_tile<256, 256, 2, 4, 2>(p, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace iqp
