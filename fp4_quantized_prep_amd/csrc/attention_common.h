// Shared by the two attention kernels: operand types, the widening of cache
// codes, and what a workgroup needs of its sequence.
#pragma once

#include "layer_common.h"

namespace iqp {
namespace {
namespace attn {

using namespace layer;

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int UNIT = 64;             // tokens the kernels take at a time
constexpr float LOWEST = -3.402823466e38f;   // no score lies below: the running maximum before the first token
// Weights are computed times a power of two, so that the largest that may occur is
// 2^FP16_TOP: fp16 then holds those far below it as well as it can.
constexpr float FP16_TOP = 15.f;

// eight E4M3 codes as bf16 / fp16: exact, without their block's scale
__device__ __forceinline__ v8bf widen_bf16(uint32_t a, uint32_t b) {
  const v2bf x0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, false), x1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, true);
  const v2bf x2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, false), x3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, true);
  return v8bf{x0[0], x0[1], x1[0], x1[1], x2[0], x2[1], x3[0], x3[1]};
}

__device__ __forceinline__ v8h widen_f16(uint32_t a, uint32_t b) {
  const v2h x0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.f, false), x1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.f, true);
  const v2h x2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.f, false), x3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.f, true);
  return v8h{x0[0], x0[1], x1[0], x1[1], x2[0], x2[1], x3[0], x3[1]};
}

// 16 bytes with those of tokens outside [lo, hi) cleared (byte j: token j)
__device__ __forceinline__ v4u clear_outside(v4u v, int lo, int hi) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int a = min(max(lo - 4 * j, 0), 4), b = min(max(hi - 4 * j, 0), 4);
    const uint32_t ma = a >= 4 ? 0u : 0xFFFFFFFFu << (8 * a);
    const uint32_t mb = b >= 4 ? 0xFFFFFFFFu : (1u << (8 * b)) - 1u;
    v[j] &= ma & mb;
  }
  return v;
}

// 1 / sum of a row's weights: 0 where it saw nothing, NaN kept
__device__ __forceinline__ float inverse_sum(float sum) { return sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum); }

// the most tokens that a row can see
inline int64_t reach(const AttnArgs& p) {
  const int64_t held = (int64_t)p.seq.max_blocks << p.seq.log_block;
  return p.window > 0 && p.window < held ? p.window : held;
}

// Where row `row` (token-major: token * group + query head of the group) of key
// head `head` lies in q and out: element offset for row stride ld.
__device__ __forceinline__ int64_t row_offset(int64_t begin, int64_t row, int head, int group, int D, int64_t ld) {
  const int64_t i = row / group;
  return (begin + i) * ld + ((int64_t)head * group + (row - i * group)) * D;
}

// Joining partial results (max, sum and unnormalised output of a row, each
// relative to its own max). A group of D / 4 lanes sums up those of a row: all of
// them where they are few (every group then has a row of its own), else every
// JOIN-th, and the groups meet in LDS.
constexpr int JOIN_THREADS = 256;
template <int D>
constexpr int join_groups() { return JOIN_THREADS / (D / 4); }

template <int D>
struct JoinSpace {
  float m[join_groups<D>()], l[join_groups<D>()];
  float o[join_groups<D>()][D];
};

struct RowSum {
  float m, l;
  v4f o;
};

// part(first), part(first + step), ... below part(n), dims d .. d + 3 of row r;
// AHEAD at a time, all loaded before the first is used
template <class Part>
__device__ __forceinline__ RowSum sum_partials(const Part& part, int first, int step, int n, int r, int d) {
  constexpr int AHEAD = 8;
  RowSum s = {LOWEST, 0.f, v4f{0.f, 0.f, 0.f, 0.f}};
  for (int w = first; w < n; w += AHEAD * step) {
    float m[AHEAD], l[AHEAD];
    v4f v[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      m[i] = LOWEST;
      l[i] = 0.f;
      v[i] = v4f{0.f, 0.f, 0.f, 0.f};
      if (w + i * step < n) {
        const auto& x = part(w + i * step);
        m[i] = x.m[r];
        l[i] = x.l[r];
        v[i] = *reinterpret_cast<const v4f*>(&x.o[r][d]);
      }
    }
    float mn = s.m;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) mn = fmaxf(mn, m[i]);
    const float b = __builtin_amdgcn_exp2f(s.m - mn);
    s.m = mn;
    s.l *= b;
#pragma unroll
    for (int j = 0; j < 4; ++j) s.o[j] *= b;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const float a = __builtin_amdgcn_exp2f(m[i] - mn);
      s.l += l[i] * a;
#pragma unroll
      for (int j = 0; j < 4; ++j) s.o[j] += v[i][j] * a;
    }
  }
  return s;
}

// Rows r0, r0 + step, ... < rows of n partial results part(0 .. n - 1);
// finish(r, d, l, o) gets a row's sum and dims d .. d + 3 of its output
template <int D, class Part, class Finish>
__device__ __forceinline__ void join_rows(JoinSpace<D>& lds, int r0, int step, int rows, int n, const Part& part, const Finish& finish) {
  constexpr int LANES = D / 4, JOIN = join_groups<D>();
  const int g = threadIdx.x / LANES, d = 4 * (threadIdx.x % LANES);
  if (n <= 8) {
    for (int r = r0 + step * g; r < rows; r += step * JOIN) {
      const RowSum s = sum_partials(part, 0, 1, n, r, d);
      finish(r, d, s.l, s.o);
    }
    return;
  }
  for (int r = r0; r < rows; r += step) {
    RowSum s = sum_partials(part, g, JOIN, n, r, d);
    if (d == 0) {
      lds.m[g] = s.m;
      lds.l[g] = s.l;
    }
    *reinterpret_cast<v4f*>(&lds.o[g][d]) = s.o;
    __syncthreads();
    if (g == 0) {
      s.m = lds.m[0];
#pragma unroll
      for (int i = 1; i < JOIN; ++i) s.m = fmaxf(s.m, lds.m[i]);
      s.l = 0.f;
      s.o = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < JOIN; ++i) {
        const float a = __builtin_amdgcn_exp2f(lds.m[i] - s.m);
        s.l += lds.l[i] * a;
        const v4f v = *reinterpret_cast<const v4f*>(&lds.o[i][d]);
#pragma unroll
        for (int j = 0; j < 4; ++j) s.o[j] += v[j] * a;
      }
      finish(r, d, s.l, s.o);
    }
    __syncthreads();
  }
}

}  // namespace attn
}  // namespace
}  // namespace iqp
