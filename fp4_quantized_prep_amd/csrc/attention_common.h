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
constexpr float LOWEST = -1e30f;     // below every score: the running maximum before the first token

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

// Where row `row` (token-major: token * group + query head of the group) of key
// head `head` lies in q and out: element offset for row stride ld.
__device__ __forceinline__ int64_t row_offset(int64_t begin, int64_t row, int head, int group, int D, int64_t ld) {
  const int64_t i = row / group;
  return (begin + i) * ld + ((int64_t)head * group + (row - i * group)) * D;
}

}  // namespace attn
}  // namespace
}  // namespace iqp
