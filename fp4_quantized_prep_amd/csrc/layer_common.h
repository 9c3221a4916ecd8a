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

// A row offset of the batch, kept inside its T rows whatever cu holds.
__device__ __forceinline__ int clamp_row(const SeqBatch& b, int v) { return v < 0 ? 0 : (v > (int)b.T ? (int)b.T : v); }

// A sequence: its rows begin .. end - 1 of the batch, and its length with them.
struct SeqRows {
  int s, begin, end, len;
};

// sequence s0 + lane of the batch (s = S and no rows past the last); one round
// of loads
__device__ __forceinline__ SeqRows lane_sequence(const SeqBatch& b, int s0) {
  const int s = s0 + (int)(threadIdx.x & 63), c = s < b.S ? s : b.S - 1;
  const int begin = b.cu[c], end = b.cu[c + 1], len = b.lens[c];
  SeqRows q = {s < b.S ? s : b.S, clamp_row(b, begin), clamp_row(b, end), len};
  if (s >= b.S) q.end = q.begin;
  return q;
}

// lane's copy of v
__device__ __forceinline__ SeqRows sequence_of_lane(const SeqRows& v, int lane) {
  return {__builtin_amdgcn_readlane(v.s, lane), __builtin_amdgcn_readlane(v.begin, lane),
          __builtin_amdgcn_readlane(v.end, lane), __builtin_amdgcn_readlane(v.len, lane)};
}

// The sequence whose range of work items holds `item`, where sequence s owns
// the items from key(s) = floor(begin(s) * mul / 2^shift) + slots * s up to
// key(s + 1). Since floor(a + b) >= floor(a) + floor(b), a sequence of n rows
// owns at least floor(n mul / 2^shift) + slots items, so the grid needs only
// the total number of rows and of sequences, and no prefix sum over the
// sequences' own counts. Every wave looks at 64 sequences at once and gets the
// same answer (S >= 1): two rounds of loads find one of 4096 (64 by 64, a token each
// for 1000 sequences took 18.5 us to append, 11.6 so; for 3000 82, 24).
__device__ __forceinline__ int64_t item_key(const SeqRows& q, int mul, int shift, int slots) {
  return (((int64_t)q.begin * mul) >> shift) + (int64_t)slots * q.s;
}

__device__ __forceinline__ SeqRows find_sequence(const SeqBatch& b, int64_t item, int mul, int shift, int slots) {
  SeqRows found = {0, 0, 0, 0};
  // of more than 64 sequences the 64th part in which it lies, until 64 are left
  int s0 = 0, count = b.S;
  while (count > 64) {
    const int step = (int)(((int64_t)count + 63) / 64), lane = threadIdx.x & 63;
    const bool in = (int64_t)lane * step < count;
    const int s = in ? s0 + lane * step : s0;
    const SeqRows q = {s, clamp_row(b, b.cu[s]), 0, 0};
    const int n = __popcll(__ballot(in && item_key(q, mul, shift, slots) <= item));
    if (n == 0) return found;
    const int skip = (n - 1) * step;
    s0 += skip;
    count = count - skip < step ? count - skip : step;
  }
  const SeqRows q = lane_sequence(b, s0);
  const int n = __popcll(__ballot(q.s < s0 + count && item_key(q, mul, shift, slots) <= item));
  if (n > 0) found = sequence_of_lane(q, n - 1);
  return found;
}

}  // namespace layer
}  // namespace
}  // namespace iqp
