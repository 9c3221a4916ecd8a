// Block-scaled FP8 products of rows sorted by group, each group with weights of
// its own (the experts of a mixture). For place i, in group g,
//   y[i, n] = sum_j 2^(ea(src, j) + ew(g, n / 128, j)) sum_{k in block j} A[src, k] W[g, n, k]
// with src = i, or the token that place i came from. The matrix cores apply the scales
// and add 64 products at a time at a fixed precision below the largest of them, which
// costs such a sum up to 2^-11.3 of that product (2^-14.5 as a rule), then add the sums
// in float32. All their FP8 forms do; as bf16 the products would go at half the rate.
// Then either
//   out = bf16(y), or, the weights' rows being I gates and I ups,
//   h[i, c] = y_c / (1 + exp(-y_c)) y_(I + c), quantised in 1x128 blocks as
//   fp8_quant_1x128_ue8m0 does, from the float32 values.
//
// A workgroup computes 256 weight rows (128 gates and their 128 ups, so that it
// holds whole blocks of h) of one tile of at most 256 places. The host knows
// neither how many rows a group has nor which groups have any, so every workgroup
// looks its tile up in the offsets, and the body goes by the tile's rows: up to 16
// the weights are streamed past them, each wave on its own; up to 64, 128, 192 and
// 256 tiles of matrix-core products whose waves share operands in LDS.
//
// Up to about 32 rows a group the read of the weights bounds it (64 groups of 4096 x
// 7168, 16 rows each: 313 us, 6.0 TB/s; 32: 319; 64: 328; 8 rows in 8 groups of 7168 x
// 2048: 20 us, 5.8). Above, neither the read nor the products alone, but part of their
// sum: 16384 rows in 64 groups 600 us, 37056 1.05 ms, 2.0 PFLOP/s; of 768 rows each
// 2.3; the same with one group's weights for all 2.7, with zeros for a 2.55, with both
// 3.05: the card lowers its clock under these products, and weights from memory cost a
// seventh of the time. The matrix cores are busy for 60 % of a CU's time and the CUs for 86 %
// (tiles of unequal length end unevenly), but the clock gives back most of what
// evenness would save. What did not help there: tiles of a group as even as can be and
// the groups sorted by them (64 groups of 4096 x 7168: 1024 tokens 457 to 428 us, but
// 4632 the same, and at 7168 x 2048 600 to 625); offsets and addresses ahead of the copies,
// so that fewer instructions stand between two MFMAs (1050 to 1081); stages of half a
// block, four deep (requests of 64 bytes: 4 % more); weights asked into L2 two blocks
// ahead (4 %); a third stage for the weights of the 192-row tile; K blocks in another
// order for each workgroup; eight waves of 64 x 128 instead of four of 128 x 128 (512
// tokens: 387 us for 367). A K of 2048 leaves 7 us of a tile's 40 to its first loads and
// its stores.
#include <type_traits>

#include "iq_common.h"
#include "layer_common.h"
#include "row_groups.h"

namespace iqp {
namespace {

enum Epilogue { TO_BF16, SWIGLU };

constexpr int SLAB = 1024;   // bytes of one wave-wide copy to LDS
constexpr int TN = 256;      // weight rows of a workgroup (SWIGLU: 128 gates and their 128 ups)
constexpr int NW = 4;        // its waves
constexpr int WN = NW / 2;   // waves along the weight rows in the tile body, two along the places
constexpr int AN = TN / 32 / WN;   // 32-row tiles of a wave there (SWIGLU: half of them gates)
constexpr int RT = TN / 16 / NW;   // 16-row tiles of a wave in the stream body (likewise)

constexpr int waitcnt_vm(int n) { return (n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14); }

// An offset beyond every buffer: operands reach less than 2^31 bytes. Joined to
// others by "or", so that two of them stay one.
constexpr uint32_t PAST = 0x80000000u;

// Rows of a that C of a lane's places read, PAST where there is none; `place(i)` is
// the i-th one's number in the tile. All entries are asked for before one is waited for,
// and `meanwhile` is done in between.
template <int C, typename Place, typename Meanwhile>
__device__ __forceinline__ void source_rows(const Fp8GroupedArgs& p, const groups::Tile& t, Place place, uint32_t (&src)[C], Meanwhile meanwhile) {
  int entry[C];
  if (p.top) {
#pragma unroll
    for (int i = 0; i < C; ++i) entry[i] = p.groups.rows[t.begin + (place(i) < t.rows ? place(i) : 0)];
    __builtin_amdgcn_sched_barrier(0);
    meanwhile();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < C; ++i) entry[i] = entry[i] < 0 ? -1 : (int)((unsigned)entry[i] / (unsigned)p.top);
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) entry[i] = t.begin + place(i);
    meanwhile();
  }
#pragma unroll
  for (int i = 0; i < C; ++i) src[i] = place(i) < t.rows && entry[i] >= 0 && entry[i] < p.M ? (uint32_t)entry[i] : PAST;
}

// what the bodies read of a group's weights
struct Weights {
  const uint8_t* base[2];    // TO_BF16: 256 rows from n0 on, twice; SWIGLU: 128 gates, 128 ups
  uint64_t bytes;            // of each
  const uint8_t* scales;     // of the group
  int64_t n0;                // first row (SWIGLU: first channel)
};

template <Epilogue EPI>
__device__ __forceinline__ Weights weights_of(const Fp8GroupedArgs& p, const groups::Tile& t) {
  Weights w;
  const uint8_t* const base = p.w + t.group * p.ldwg;
  w.scales = p.w_scales + t.group * p.ld_wsg;
  w.n0 = (int64_t)t.part * (EPI == SWIGLU ? TN / 2 : TN);
  const int64_t rows = EPI == SWIGLU ? TN / 2 : p.N - w.n0 < TN ? p.N - w.n0 : TN;
  w.base[0] = base + w.n0 * p.ldw;
  w.base[1] = EPI == SWIGLU ? base + (p.N / 2 + w.n0) * p.ldw : w.base[0];
  w.bytes = (uint64_t)(rows - 1) * p.ldw + (uint64_t)KB * p.nkb;
  return w;
}

// The scale bytes of 128-row tile `tile` of the group's weights, 4 K blocks a lane:
// asked for before the first copies, put together behind them.
struct ScaleBytes {
  uint8_t b[4];
  __device__ __forceinline__ uint32_t lanes() const { return b[0] | b[1] << 8 | b[2] << 16 | (uint32_t)b[3] << 24; }
};

__device__ __forceinline__ ScaleBytes scale_bytes(const Fp8GroupedArgs& p, const Weights& w, int64_t tile, int lane) {
  const int64_t last = (p.N + 127) / 128 - 1;
  const uint8_t* const s = w.scales + (tile < last ? tile : last) * p.ld_ws;
  ScaleBytes v;
#pragma unroll
  for (int b = 0; b < 4; ++b) v.b[b] = s[4 * lane + b < p.nkb ? 4 * lane + b : 0];
  return v;
}

__device__ __forceinline__ int scale_of(uint32_t lanes, int j) {
  return (int)((uint32_t)__builtin_amdgcn_readlane((int)lanes, (j >> 2) & 63) >> (8 * (j & 3)));
}

// gate / (1 + e^-gate) up to float32's own roundings. e^-gate = 2^(t + r): t the
// product with 1 / ln 2 as rounded, r what that rounding and the constant's left out
// (up to 2^-18 of the exponent), 2^r = 1 + r ln 2. Where 2^t is 0 or infinite the correction may be no
// number, and the maximum takes the other. Then a quarter of the quotient's two sides,
// as the reciprocal of a number beyond 2^126 is 0, by reciprocal and correction. (1024
// tokens of 64 experts, K 512 / 7168, us: so 61.7 / 442, with expf and a division 70.0 /
// 448, without the correction and with a division 61.2 / 441.)
__device__ __forceinline__ float swiglu(float gate, float up) {
  const float t = gate * -1.44269502f;
  const float r = __builtin_fmaf(gate, -1.92596299e-8f, __builtin_fmaf(gate, -1.44269502f, -t));
  const float e0 = __builtin_amdgcn_exp2f(t);
  const float e = __builtin_fmaxf(__builtin_fmaf(e0, r * 0.693147181f, e0), e0 * 0.999f);
  const float n = 0.25f * gate, d = __builtin_fmaf(e, 0.25f, 0.25f), i = __builtin_amdgcn_rcpf(d);
  const float q = n * i;
  return __builtin_amdgcn_div_fixupf(__builtin_fmaf(__builtin_fmaf(-d, q, n), i, q), d, n) * up;
}

// The exponent of a block from its largest magnitude (float32 bits): the least
// e >= -22 with 448 2^e >= amax. amax = (1 + f 2^-23) 2^(E - 127), 448 = 1.75 2^8.
__device__ __forceinline__ int exponent_of(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 135 + ((b & 0x7FFFFF) > 0x600000 ? 1 : 0);
  return e > -22 ? e : -22;
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float mul) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a * mul, b * mul, 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(c * mul, d * mul, r, true);
  return (uint32_t)r;
}

// scale byte of channels n0 .. n0 + 127 of a place; the last one's word is filled up with zeros
__device__ __forceinline__ void store_scale(const Fp8GroupedArgs& p, int64_t place, int64_t n0, int e) {
  const int block = (int)(n0 / 128), blocks = (int)(p.N / 256);
  uint8_t* const word = reinterpret_cast<uint8_t*>(p.q_scales + place * p.qs_sm + (int64_t)(block >> 2) * p.qs_sw);
  word[block & 3] = (uint8_t)(e + 127);
  if (block == blocks - 1)
    for (int b = (block & 3) + 1; b < 4; ++b) word[b] = 0;
}

// Tile body: 256 weight rows x up to TM = 64 AM places, four waves of 128 x 32 AM
// (2 by 2; the places in tiles of 32 that alternate between the two). K block by
// K block through NST LDS stages, 8 rows of 128 bytes a copy, the 16-byte chunks
// of LDS row r permuted by (r / 2) % 8 so that the operand reads meet distinct
// banks; weight row n of a 32-row tile sits in LDS row 8 ((n / 4) % 4) + 4 (n / 16)
// + n % 4 of it, so that a lane's sixteen accumulators are sixteen consecutive n
// of one place. Copies past the last block or row read zeros out of bounds,
// which keeps the wait counts constant.
template <int AM, int NST>
constexpr int tile_bytes() { return NST * (TN * KB + 64 * AM * (KB + 4)); }

template <Epilogue EPI, int AM, int NST>
__device__ __forceinline__ void tile_body(const Fp8GroupedArgs& p, const groups::Tile& t, uint8_t* lds) {
  constexpr int TM = 64 * AM;
  constexpr int W_BYTES = TN * KB, A_BYTES = TM * KB, S_BYTES = TM * 4;
  constexpr int WC = W_BYTES / SLAB / NW, AC = A_BYTES / SLAB / NW, NCOPY = WC + AC + 1;
  static_assert(WC * NW * SLAB == W_BYTES && AC * NW * SLAB == A_BYTES && WC % 2 == 0, "whole slabs");
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave % WN, wm = wave / WN;
  uint8_t* const lw = lds;
  uint8_t* const la = lw + NST * W_BYTES;
  uint8_t* const ls = la + NST * A_BYTES;
  const Weights w = weights_of<EPI>(p, t);
  const int nkb = p.nkb;
  const int64_t nw = (nkb + 3) / 4;
  const uint64_t a_bytes = (uint64_t)(p.M - 1) * p.lda + (uint64_t)KB * nkb;
  const uint64_t s_bytes = 4 * (uint64_t)((p.M - 1) * p.as_sm + (nw - 1) * p.as_sw + 1);

  // copies: slab i of this wave is LDS rows 8 (wave + NW i) + lane / 8
  uint32_t vw[WC], va[AC], vs;
#pragma unroll
  for (int i = 0; i < WC; ++i) {
    int r = 8 * (wave + NW * i) + (lane >> 3);
    const int chunk = 16 * ((lane & 7) ^ ((r >> 1) & 7));
    if (EPI == SWIGLU) r &= TN / 2 - 1;
    const int n = (r & ~31) + 4 * ((r >> 3) & 3) + 16 * ((r >> 2) & 1) + (r & 3);
    vw[i] = (uint32_t)(n * (int)p.ldw + chunk);
  }

  // Copy c (0 .. NCOPY - 1) of block j into stage st. Past the last block the buffers
  // are of no bytes: the copies read zeros, with the offset left at 0.
  auto copy = [&](int j, int st, int c) __attribute__((always_inline)) {
    const bool in = j < nkb;
    const int at = in ? KB * j : 0;
    if (c < WC) {
      const int h = c / (WC / 2);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(w.base[h], in ? w.bytes : 0), (lds_void*)(lw + st * W_BYTES + SLAB * (wave + NW * c)),
                                               16, vw[c], at, 0, 0);
    } else if (c < WC + AC) {
      const int k = c - WC;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(p.a, in ? a_bytes : 0), (lds_void*)(la + st * A_BYTES + SLAB * (wave + NW * k)), 16,
                                               va[k], at, 0, 0);
    } else {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(p.a_scales, in ? s_bytes : 0), (lds_void*)(ls + st * S_BYTES + 256 * (wave % AM)), 4,
                                               vs, in ? 4 * (j >> 2) * (int)p.as_sw : 0, 0, 0);
    }
  };

  // the weight scales of the first and the second half of the wave's rows
  const ScaleBytes wb0 = scale_bytes(p, w, (w.n0 + (EPI == SWIGLU ? 0 : 32 * AN * wn)) / 128, lane);
  const ScaleBytes wb1 = EPI == SWIGLU ? scale_bytes(p, w, (p.N / 2 + w.n0) / 128, lane) : wb0;
  // (the first block's weights go ahead of the rows: 37056 of them, K 2048, 601 to 590 us)
  uint32_t src[AC + 1];
  const auto place = [&](int i) __attribute__((always_inline)) { return i < AC ? 8 * (wave + NW * i) + (lane >> 3) : 64 * (wave % AM) + lane; };
  source_rows(p, t, place, src, [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < WC; ++c) copy(0, 0, c);
  });
#pragma unroll
  for (int i = 0; i < AC; ++i) va[i] = src[i] == PAST ? PAST : src[i] * (uint32_t)p.lda + 16 * ((lane & 7) ^ ((place(i) >> 1) & 7));
  vs = src[AC] == PAST ? PAST : 4 * src[AC] * (uint32_t)p.as_sm;
#pragma unroll
  for (int i = 0; i < NST; ++i)
#pragma unroll
    for (int c = i ? 0 : WC; c < NCOPY; ++c) copy(i, i, c);
  __builtin_amdgcn_sched_barrier(0);
  const uint32_t wsc0 = wb0.lanes(), wsc1 = EPI == SWIGLU ? wb1.lanes() : wsc0;

  v16f acc[AN][AM];
#pragma unroll
  for (int i = 0; i < AN; ++i)
#pragma unroll
    for (int j = 0; j < AM; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // Half-steps of 64 columns. The next half's operands are read while this one's are
  // multiplied: the weights' into registers of their own, the places' one by one as
  // the MFMAs are done with them. One barrier a block, behind the first MFMAs of its
  // second half: by then every wave has read all of block j, whose stage is refilled,
  // and block j + 1 has landed (only the NST - 2 blocks after it may be in flight).
  // With one wave a SIMD, what is not an MFMA has to fit beside one: reads and copies
  // go between the MFMAs one at a time, and offsets are scalar (37056 rows, 4096 x 7168: 1164 to 1099 us, 7168 x
  // 2048: 644 to 605).
  constexpr int WAIT = waitcnt_vm((NST - 2) * NCOPY);
  const int row = lane & 31, swz = (row >> 1) & 7;
  v8i fw[2][AN], fa[AM];
  uint32_t as_word[AM];
  auto read = [&](const uint8_t* b, int kh) __attribute__((always_inline)) {
    const int c0 = 16 * ((4 * kh + 2 * half) ^ swz), c1 = 16 * ((4 * kh + 2 * half + 1) ^ swz);
    return make_v8i(*reinterpret_cast<const v4u*>(b + c0), *reinterpret_cast<const v4u*>(b + c1));
  };
  auto read_a = [&](int st, int kh, int u) __attribute__((always_inline)) {
    fa[u] = read(la + st * A_BYTES + KB * (32 * (2 * u + wm) + row), kh);
  };
  auto read_w = [&](int st, int kh, int i) __attribute__((always_inline)) {
    const int r = EPI == SWIGLU ? 128 * (i / (AN / 2)) + 32 * (AN / 2 * wn + i % (AN / 2)) : 32 * (AN * wn + i);
    fw[kh][i] = read(lw + st * W_BYTES + KB * (r + row), kh);
  };
  auto read_scale = [&](int st, int u) __attribute__((always_inline)) {
    as_word[u] = *reinterpret_cast<const uint32_t*>(ls + st * S_BYTES + 4 * (32 * (2 * u + wm) + row));
  };
  {
    constexpr int FIRST = waitcnt_vm((NST - 1) * NCOPY);
    __builtin_amdgcn_s_waitcnt(FIRST);
  }
  block_barrier();
#pragma unroll
  for (int i = 0; i < AN; ++i) read_w(0, 0, i);
#pragma unroll
  for (int u = 0; u < AM; ++u) {
    read_scale(0, u);
    read_a(0, 0, u);
  }
  int st = 0;
  for (int j = 0; j < nkb; ++j) {
    const int st1 = st + 1 < NST ? st + 1 : 0;
    const int ws[2] = {scale_of(wsc0, j), scale_of(wsc1, j)};
    int as[AM];
#pragma unroll
    for (int u = 0; u < AM; ++u) {
      as[u] = (int)(as_word[u] >> (8 * (j & 3)));
#pragma unroll
      for (int i = 0; i < AN; ++i) {
        acc[i][u] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fw[0][i], fa[u], acc[i][u], 0, 0, 0, ws[i / (AN / 2)], 0, as[u]);
        __builtin_amdgcn_sched_barrier(0);
        if (u == 0) read_w(st, 1, i);
        if (i == AN - 1) read_a(st, 1, u);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    // the slots behind the MFMAs of the second half, but for the first one's
    constexpr int SLOTS = AN * AM - 1;
#pragma unroll
    for (int u = 0; u < AM; ++u)
#pragma unroll
      for (int i = 0; i < AN; ++i) {
        acc[i][u] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fw[1][i], fa[u], acc[i][u], 0, 0, 0, ws[i / (AN / 2)], 0, as[u]);
        __builtin_amdgcn_sched_barrier(0);
        const int slot = u * AN + i - 1;
        if (slot == 0) {
          __builtin_amdgcn_s_waitcnt(WAITCNT_LGKM0);
          __builtin_amdgcn_s_waitcnt(WAIT);
          block_barrier();
        }
        if (slot >= 0) {
#pragma unroll
          for (int c = NCOPY * slot / SLOTS; c < NCOPY * (slot + 1) / SLOTS; ++c) copy(j + NST, st, c);
#pragma unroll
          for (int k = AN * slot / SLOTS; k < AN * (slot + 1) / SLOTS; ++k) read_w(st1, 0, k);
          if (i == AN - 1) {
            read_scale(st1, u);
            read_a(st1, 0, u);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    st = st1;
  }

  // in the ring's place: every wave has read its operands, and no copy is in flight
  __builtin_amdgcn_s_waitcnt(WAITCNT_VM0);
  __syncthreads();
  if constexpr (EPI == SWIGLU) {
    float* const amax = reinterpret_cast<float*>(lds);    // [wn][TM]
#pragma unroll
    for (int u = 0; u < AM; ++u) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < AN / 2; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          acc[i][u][r] = swiglu(acc[i][u][r], acc[AN / 2 + i][u][r]);
          m = fmaxf(m, fabsf(acc[i][u][r]));
        }
      m = fmaxf(m, __shfl_xor(m, 32));
      if (half == 0) amax[wn * TM + 32 * (2 * u + wm) + row] = m;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < AM; ++u) {
      const int r = 32 * (2 * u + wm) + row;
      float m = amax[r];
#pragma unroll
      for (int v = 1; v < WN; ++v) m = fmaxf(m, amax[v * TM + r]);
      const int e = exponent_of(m);
      const float mul = layer::pow2(-e);
      if (r < t.rows) {
        const int64_t place = t.begin + r;
#pragma unroll
        for (int i = 0; i < AN / 2; ++i) {
          const v16f& h = acc[i][u];
          uint32_t d[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) d[k] = codes4(h[4 * k], h[4 * k + 1], h[4 * k + 2], h[4 * k + 3], mul);
          *reinterpret_cast<v4u*>(p.q + place * p.ldq + w.n0 + 32 * (AN / 2 * wn + i) + 16 * half) = v4u{d[0], d[1], d[2], d[3]};
        }
        if (wn == 0 && half == 0) store_scale(p, place, w.n0, e);
      }
    }
  } else {
    // through the wave's part of LDS, 32 places at a time, so that a store covers
    // whole stretches of a row, 16 bytes a lane whatever its alignment; a row's last
    // columns, fewer than eight, go one by one
    constexpr int PITCH = 64 * AN + 16, LANES = 4 * AN;   // bytes of a place's row; 16-byte pieces of it
    uint8_t* const mine = lds + wave * 32 * PITCH;
    const int64_t n0 = w.n0 + 32 * AN * wn;
    const int rows_n = p.N - n0 < 32 * AN ? (int)(p.N - n0) : 32 * AN;
#pragma unroll
    for (int u = 0; u < AM; ++u) {
      const int m = 32 * (2 * u + wm);
      const int rows_m = t.rows - m < 32 ? t.rows - m : 32;
#pragma unroll
      for (int i = 0; i < AN; ++i) {
        uint32_t d[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) d[r] = layer::pack_bf16(acc[i][u][2 * r], acc[i][u][2 * r + 1]);
        uint8_t* const to = mine + row * PITCH + 64 * i + 32 * half;
        *reinterpret_cast<v4u*>(to) = v4u{d[0], d[1], d[2], d[3]};
        *reinterpret_cast<v4u*>(to + 16) = v4u{d[4], d[5], d[6], d[7]};
      }
      asm volatile("" ::: "memory");   // the wave's own writes, then its own reads: in order
      uint16_t* const to = p.out + (int64_t)(t.begin + m) * p.ldo + n0;
#pragma unroll
      for (int i = 0; i < 32; i += 64 / LANES) {
        const int r = i + lane / LANES, c = 8 * (lane % LANES);
        const v4u v = *reinterpret_cast<const v4u*>(mine + r * PITCH + 2 * c);
        if (r < rows_m) {
          if (c + 8 <= rows_n) {
            if (p.stream_out) __builtin_nontemporal_store(v, reinterpret_cast<groups::v4u_any*>(to + r * p.ldo + c));
            else *reinterpret_cast<groups::v4u_any*>(to + r * p.ldo + c) = v;
          } else
            for (int e = 0; c + e < rows_n; ++e) to[r * p.ldo + c + e] = *reinterpret_cast<const uint16_t*>(mine + r * PITCH + 2 * (c + e));
        }
      }
      asm volatile("" ::: "memory");
    }
  }
}

// Stream body, for up to 16 MT places: the product is then a read of the
// weights. Each wave owns 64 of the workgroup's 256 rows (SWIGLU: 32 gates and
// their 32 ups) and walks all K blocks with an LDS ring of its own: no barrier
// in the loop, only the wave's wait counts. 16x16x128 MFMA: weight rows as its
// rows, places as its columns. Workgroups start the K blocks at different
// places, as all rows lie at equal strides and would share memory channels.
template <int MT>
constexpr int stream_stage() { return (16 * RT + 16 * MT) * KB + 256; }

template <Epilogue EPI, int MT, int NST>
__device__ __forceinline__ void stream_body(const Fp8GroupedArgs& p, const groups::Tile& t, uint8_t* lds) {
  constexpr int TOK = 16 * MT, STAGE = stream_stage<MT>();
  constexpr int WR = 16 * RT, WC = WR / 8, AC = TOK / 8, NCOPY = WC + AC + 1;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Weights w = weights_of<EPI>(p, t);
  const int nkb = p.nkb;
  const rsrc_t rw[2] = {make_rsrc(w.base[0], w.bytes), make_rsrc(w.base[1], w.bytes)};
  const int rot = (int)((unsigned)(t.part * 5 + t.group * 3) % (unsigned)nkb);
  const int64_t nw = (nkb + 3) / 4;
  const rsrc_t ra = make_rsrc(p.a, (uint64_t)(p.M - 1) * p.lda + (uint64_t)KB * nkb);
  const rsrc_t rs = make_rsrc(p.a_scales, 4 * (uint64_t)((p.M - 1) * p.as_sm + (nw - 1) * p.as_sw + 1));
  // copy c moves rows 8 c + lane / 8, 16-byte chunk permuted by (row / 2) % 8
  uint32_t vw[WC], va[AC];
#pragma unroll
  for (int c = 0; c < WC; ++c) {
    const int r = 8 * c + (lane >> 3);
    const int n = EPI == SWIGLU ? WR / 2 * wave + r % (WR / 2) : WR * wave + r;
    vw[c] = (uint32_t)(n * (int)p.ldw + 16 * ((lane & 7) ^ ((r >> 1) & 7)));
  }
  uint32_t src[AC + 1];
  const auto place = [&](int i) __attribute__((always_inline)) { return i < AC ? 8 * i + (lane >> 3) : lane; };
  source_rows(p, t, place, src, [] {});
#pragma unroll
  for (int c = 0; c < AC; ++c) va[c] = src[c] == PAST ? PAST : src[c] * (uint32_t)p.lda + 16 * ((lane & 7) ^ ((place(c) >> 1) & 7));
  const uint32_t vs = src[AC] == PAST ? PAST : 4 * src[AC] * (uint32_t)p.as_sm;
  uint8_t* const ring = lds + wave * NST * STAGE;

  // the i-th block of the walk into stage st
  auto block_of = [&](int i) __attribute__((always_inline)) { return i + rot < nkb ? i + rot : i + rot - nkb; };
  auto copy = [&](int i, int st) __attribute__((always_inline)) {
    const int j = block_of(i);
    const uint32_t past = i < nkb ? 0 : PAST, u = KB * j;
    uint8_t* const b = ring + st * STAGE;
#pragma unroll
    for (int c = 0; c < WC; ++c)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw[c / (WC / 2)], (lds_void*)(b + SLAB * c), 16, (vw[c] + u) | past, 0, 0, 0);
#pragma unroll
    for (int c = 0; c < AC; ++c)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(b + WR * KB + SLAB * c), 16, (va[c] + u) | past, 0, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(b + (WR + TOK) * KB), 4, (vs + 4 * (j >> 2) * (int)p.as_sw) | past, 0, 0, 0);
  };

  const ScaleBytes wb0 = scale_bytes(p, w, (w.n0 + (EPI == SWIGLU ? 0 : WR * wave)) / 128, lane);
  const ScaleBytes wb1 = EPI == SWIGLU ? scale_bytes(p, w, (p.N / 2 + w.n0) / 128, lane) : wb0;
#pragma unroll
  for (int st = 0; st < NST; ++st) copy(st, st);
  __builtin_amdgcn_sched_barrier(0);
  const uint32_t wsc0 = wb0.lanes(), wsc1 = EPI == SWIGLU ? wb1.lanes() : wsc0;

  v4f acc[RT][MT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m] = v4f{0.f, 0.f, 0.f, 0.f};
  constexpr int WAIT = waitcnt_vm((NST - 1) * NCOPY);
  const int swz = (col >> 1) & 7;
  const int c0 = 16 * ((2 * g) ^ swz), c1 = 16 * ((2 * g + 1) ^ swz);
  int st = 0;
  for (int i = 0; i < nkb; ++i) {
    __builtin_amdgcn_s_waitcnt(WAIT);
    asm volatile("" ::: "memory");
    const int j = block_of(i);
    const uint8_t* const b = ring + st * STAGE;
    const int ws[2] = {scale_of(wsc0, j), scale_of(wsc1, j)};
    v8i fw[RT], fa[MT];
    int as[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
      as[m] = (int)(*reinterpret_cast<const uint32_t*>(b + (WR + TOK) * KB + 4 * (16 * m + col)) >> (8 * (j & 3)));
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const uint8_t* x = b + KB * (16 * r + col);
      fw[r] = make_v8i(*reinterpret_cast<const v4u*>(x + c0), *reinterpret_cast<const v4u*>(x + c1));
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const uint8_t* x = b + WR * KB + KB * (16 * m + col);
      fa[m] = make_v8i(*reinterpret_cast<const v4u*>(x + c0), *reinterpret_cast<const v4u*>(x + c1));
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
      for (int m = 0; m < MT; ++m)
        acc[r][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw[r], fa[m], acc[r][m], 0, 0, 0, ws[r / (RT / 2)], 0, as[m]);
    st = st + 1 < NST ? st + 1 : 0;
  }

  if constexpr (EPI == SWIGLU) {
    __builtin_amdgcn_s_waitcnt(WAITCNT_VM0);
    __syncthreads();
    float* const amax = reinterpret_cast<float*>(lds);    // [wave][TOK], in the rings' place
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < RT / 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          acc[i][m][r] = swiglu(acc[i][m][r], acc[RT / 2 + i][m][r]);
          x = fmaxf(x, fabsf(acc[i][m][r]));
        }
      x = fmaxf(x, __shfl_xor(x, 16));
      x = fmaxf(x, __shfl_xor(x, 32));
      if (g == 0) amax[wave * TOK + 16 * m + col] = x;
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int r = 16 * m + col;
      float x = amax[r];
#pragma unroll
      for (int v = 1; v < NW; ++v) x = fmaxf(x, amax[v * TOK + r]);
      const int e = exponent_of(x);
      if (r < t.rows) {
        const int64_t place = t.begin + r;
#pragma unroll
        for (int i = 0; i < RT / 2; ++i)
          *reinterpret_cast<uint32_t*>(p.q + place * p.ldq + w.n0 + WR / 2 * wave + 16 * i + 4 * g) =
              codes4(acc[i][m][0], acc[i][m][1], acc[i][m][2], acc[i][m][3], layer::pow2(-e));
        if (wave == 0 && g == 0) store_scale(p, place, w.n0, e);
      }
    }
  } else {
#pragma unroll
    for (int m = 0; m < MT; ++m)
      if (16 * m + col < t.rows)
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const int64_t n = w.n0 + WR * wave + 16 * r + 4 * g;
          const uint32_t lo = layer::pack_bf16(acc[r][m][0], acc[r][m][1]), hi = layer::pack_bf16(acc[r][m][2], acc[r][m][3]);
          uint16_t* const to = p.out + (int64_t)(t.begin + 16 * m + col) * p.ldo + n;
          if (n + 4 <= p.N) {
            *reinterpret_cast<groups::v2u_any*>(to) = layer::v2u{lo, hi};
          } else {
            if (n < p.N) to[0] = (uint16_t)lo;
            if (n + 1 < p.N) to[1] = (uint16_t)(lo >> 16);
            if (n + 2 < p.N) to[2] = (uint16_t)hi;
            if (n + 3 < p.N) to[3] = (uint16_t)(hi >> 16);
          }
        }
  }
}

constexpr int STREAM_LDS = NW * 3 * stream_stage<1>(), TILE_LDS = tile_bytes<2, 3>();      // 123 and 145.5 KiB
constexpr int LDS_BYTES = STREAM_LDS > TILE_LDS ? STREAM_LDS : TILE_LDS;
static_assert(LDS_BYTES >= tile_bytes<1, 3>() && LDS_BYTES >= tile_bytes<3, 2>() && LDS_BYTES >= tile_bytes<4, 2>(), "LDS");
static_assert(LDS_BYTES <= 160 * 1024 && LDS_BYTES >= NW * 32 * (64 * AN + 16), "LDS");

// Parts of a tile in a row before the next tile of the group. Workgroups go to an
// XCD's CUs by turns: with one, large tiles and their groups' remainders alternate,
// and half of the CUs get all the large ones (us, 1 / 4: 264 rows in each of 64 groups,
// 4096 x 7168 767 / 681, 7168 x 2048 419 / 351; 512 rows 871 / 874; 37056 uneven rows the
// same, 8 and 16 in a row 1 and 8 % more).
constexpr int RUN = 4;

// One tile a workgroup, by the body that its number of rows asks for: the host
// does not know how many rows a group has.
template <Epilogue EPI>
__global__ __launch_bounds__(NW * 64)
void fp8_grouped_kernel(Fp8GroupedArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[LDS_BYTES];
  const groups::Tile t = groups::find_tile(p.groups, 256, p.parts, RUN, groups::item_of(blockIdx.x, p.chunk), p.large_first);
  if (t.rows <= 0) return;
  if (t.rows <= 16) stream_body<EPI, 1, 3>(p, t, lds);
  else if (t.rows <= 64) tile_body<EPI, 1, 3>(p, t, lds);
  else if (t.rows <= 128) tile_body<EPI, 2, 3>(p, t, lds);
  else if (t.rows <= 192) tile_body<EPI, 3, 2>(p, t, lds);
  else tile_body<EPI, 4, 2>(p, t, lds);
}

}  // namespace

namespace {

// at most so many tiles: whole ones, and one that is not for every group
int64_t tiles_of(int64_t R, int32_t G) { return R / 256 + (G < R ? G : R); }

constexpr int MAX_CHUNK = 32;

}  // namespace

int64_t fp8_grouped_workgroups(int64_t R, int32_t G, int64_t N) { return tiles_of(R, G) * ((N + TN - 1) / TN) + 8 * MAX_CHUNK; }

hipError_t launch_fp8_grouped(Fp8GroupedArgs p, hipStream_t stream) {
  p.parts = (int32_t)((p.N + TN - 1) / TN);
  const int64_t items = tiles_of(p.groups.R, p.groups.G) * p.parts;
  // A CU's neighbours on its XCD share weights and rows where tiles are many (37056 rows,
  // 64 groups of 4096 x 7168: 8 to 32 in a row the same, 1 4 % more, 128 3 %); with few of
  // them every XCD has to get its part.
  p.chunk = items >= 2048 ? MAX_CHUNK : 1;
  // An output that the caches cannot keep for its reader goes past them (531 MB, K
  // 2048: 632 us for 644).
  p.stream_out = p.groups.R * p.N * 2 > ((int64_t)256 << 20);
  // Where the CUs get about two tiles each, of which some may be whole ones, the
  // large ones come first (777 tokens, 4 of 40 experts, N 2115, K 1536: 38 us for 46);
  // with more of them the search for them costs more than it gives (512 tokens, 8 of
  // 64, K 7168 366 / 376; K 2048, 8 tokens 95 / 109).
  p.large_first = items <= 512 && p.groups.R >= 16 * (int64_t)p.groups.G;
  const int64_t blocks = (items + 8 * p.chunk - 1) / (8 * p.chunk) * (8 * p.chunk);
  if (p.q)
    hipLaunchKernelGGL((fp8_grouped_kernel<SWIGLU>), dim3((unsigned)blocks), dim3(NW * 64), 0, stream, p);
  else
    hipLaunchKernelGGL((fp8_grouped_kernel<TO_BF16>), dim3((unsigned)blocks), dim3(NW * 64), 0, stream, p);
  return hipGetLastError();
}

}  // namespace iqp
