// Device helpers of the operators around an attention layer (qk_norm_rope,
// the FP8 key/value cache, attention over it): bf16 packing and the lookup of
// a workgroup's sequence in a ragged batch.
#pragma once

#include "iqp_internal.h"

namespace iqp {
namespace {
namespace layer {

typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf16_lo(uint32_t d) { return __uint_as_float(d << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t d) { return __uint_as_float(d & 0xFFFF0000u); }

// two floats as a dword of bf16, round to nearest even
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const v2bf r = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, r);
}

// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// first row of sequence s (s <= S) among the batch's T rows, kept inside them
// whatever cu holds
__device__ __forceinline__ int64_t seq_begin(const SeqBatch& b, int s) {
  const int64_t v = b.cu[s];
  return v < 0 ? 0 : (v > b.T ? b.T : v);
}

// The sequence whose range of work items holds `item`, where sequence s owns
// the items from key(s) = floor(begin(s) * mul / 2^shift) + slots * s up to
// key(s + 1). Since floor(a + b) >= floor(a) + floor(b), a sequence of n rows
// owns at least floor(n mul / 2^shift) + slots items, so the grid needs only
// the total number of rows and of sequences, and no prefix sum over the
// sequences' own counts. Every lane of a wave gets the same answer: 64
// sequences are looked at at once.
__device__ __forceinline__ int64_t item_key(const SeqBatch& b, int s, int mul, int shift, int slots) {
  return ((seq_begin(b, s) * mul) >> shift) + (int64_t)slots * s;
}

__device__ __forceinline__ int find_sequence(const SeqBatch& b, int64_t item, int mul, int shift, int slots) {
  const int lane = threadIdx.x & 63;
  int found = 0;
  for (int s0 = 0; s0 < b.S; s0 += 64) {
    const int s = s0 + lane;
    const bool below = s < b.S && item_key(b, s, mul, shift, slots) <= item;
    const int n = __popcll(__ballot(below));
    found += n;
    if (n < 64) break;
  }
  return __builtin_amdgcn_readfirstlane(found > 0 ? found - 1 : 0);
}

}  // namespace layer
}  // namespace
}  // namespace iqp
