// RMS norm of every query and key head and the rotary position embedding, in
// one pass over the projection's output.
//
// For a head x of D values at position p, with weights w:
//   y_d = x_d * rsqrt(mean(x^2) + eps) * w_d                         (float32)
//   the pairs (a, b) of the first rope_dim dims, (i, i + rope_dim / 2) or
//   (2i, 2i + 1): a' = a cos - b sin, b' = b cos + a sin, with
//   cos = table[p, i], sin = table[p, rope_dim / 2 + i]
// and one rounding to bf16 at the end.
//
// HBM-bound: 2 bytes in and 2 out per value. D / 8 consecutive lanes hold a
// head, 8 values (16 bytes) each, so a wave's load covers 64 * 16 consecutive
// bytes of a token's row; the sum of squares is reduced over those lanes with
// DPP moves. The partner of a half-split pair is rope_dim / 16 lanes away: the
// lanes exchange the four raw dwords (both halves of a pair share the norm,
// and each lane keeps its partner's weights beside its own), which costs four
// cross-lane moves a head. A wave takes PASSES groups of heads of one token,
// loads first, with the token's table row and the weights read once.
//
// Measured: 4632 tokens, 64 query and 8 key heads of 128: 36.2 us, 4.75 TB/s (a large
// copy reaches 5.1); 16 tokens: 3.0 us.
#include <type_traits>

#include "layer_common.h"

namespace iqp {
namespace {

using namespace layer;

constexpr int NORM_WAVES = 4;

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  auto dpp = [](float x, auto ctrl) __attribute__((always_inline)) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value, 0xF, 0xF, false));
  };
  v += dpp(v, std::integral_constant<int, 0xB1>{});    // lane ^ 1
  v += dpp(v, std::integral_constant<int, 0x4E>{});    // lane ^ 2
  v += dpp(v, std::integral_constant<int, 0x141>{});   // the other four of eight
  if constexpr (LANES >= 16) v += dpp(v, std::integral_constant<int, 0x140>{});   // the other eight of sixteen
  if constexpr (LANES >= 32) v += __shfl_xor(v, 16);
  return v;
}

// D values a head; PASSES groups of 64 / (D / 8) heads a wave; STREAM: loads
// and stores past the caches
template <int D, bool INTERLEAVED, int PASSES, bool STREAM>
__global__ __launch_bounds__(NORM_WAVES * 64)
void qk_norm_rope_kernel(QkNormRopeArgs p) {
  constexpr int LANES = D / 8;             // lanes of a head
  constexpr int HEADS = 64 / LANES;        // heads of a pass
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int total = p.Hq + p.Hk;
  const int per_token = (total + HEADS * PASSES - 1) / (HEADS * PASSES);   // waves of a token
  const int64_t unit = (int64_t)blockIdx.x * NORM_WAVES + wave;
  const int64_t token = unit / per_token;
  if (token >= p.M) return;                // uniform over the wave
  const int head0 = (int)(unit - token * per_token) * HEADS * PASSES + lane / LANES;
  const int l = lane % LANES;              // dims 8 l .. 8 l + 7

  v4u x[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int h = head0 + HEADS * i;
    x[i] = v4u{0u, 0u, 0u, 0u};
    if (h < total) {
      const v4u* src = reinterpret_cast<const v4u*>(h < p.Hq ? p.q + token * p.ldq + (int64_t)h * D + 8 * l
                                                             : p.k + token * p.ldk + (int64_t)(h - p.Hq) * D + 8 * l);
      x[i] = STREAM ? __builtin_nontemporal_load(src) : *src;
    }
  }

  int64_t pos = p.positions[token];
  pos = pos < 0 ? 0 : (pos >= p.max_pos ? p.max_pos - 1 : pos);
  const float* row = p.cos_sin + pos * p.rope_dim;
  const int half = p.rope_dim >> 1;
  const bool turned = 8 * l < p.rope_dim;
  const bool upper = !INTERLEAVED && 8 * l >= half;   // the second of its half-split pairs
  // the lane's angles, and its partner's lane
  constexpr int NPAIR = INTERLEAVED ? 4 : 8;
  float c[NPAIR], s[NPAIR];
#pragma unroll
  for (int i = 0; i < NPAIR; ++i) {
    c[i] = 1.f;
    s[i] = 0.f;
  }
  const int pair0 = INTERLEAVED ? 4 * l : (upper ? 8 * l - half : 8 * l);
  if (turned) {
#pragma unroll
    for (int i = 0; i < NPAIR; i += 4) {
      const v4f cc = *reinterpret_cast<const v4f*>(row + pair0 + i);
      const v4f ss = *reinterpret_cast<const v4f*>(row + half + pair0 + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c[i + j] = cc[j];
        s[i + j] = upper ? ss[j] : (INTERLEAVED ? ss[j] : -ss[j]);
      }
    }
  }
  const int shift = p.rope_dim >> 4;                  // lanes between the halves of a pair
  const int partner_l = INTERLEAVED || !turned ? l : (upper ? l - shift : l + shift);
  const int partner = lane - l + partner_l;

  // the weights of the lane's dims and of its partner's, for queries and keys
  const v4u wq = *reinterpret_cast<const v4u*>(p.q_weight + 8 * l);
  const v4u wk = *reinterpret_cast<const v4u*>(p.k_weight + 8 * l);
  v4u wq_p = wq, wk_p = wk;
  if constexpr (!INTERLEAVED) {
    wq_p = *reinterpret_cast<const v4u*>(p.q_weight + 8 * partner_l);
    wk_p = *reinterpret_cast<const v4u*>(p.k_weight + 8 * partner_l);
  }

  auto put = [&](int h, v4u out) __attribute__((always_inline)) {
    v4u* dst = reinterpret_cast<v4u*>(h < p.Hq ? p.q_out + token * p.ldqo + (int64_t)h * D + 8 * l
                                               : p.k_out + token * p.ldko + (int64_t)(h - p.Hq) * D + 8 * l);
    if constexpr (STREAM)
      __builtin_nontemporal_store(out, dst);
    else
      *dst = out;
  };
  uint64_t infinite[PASSES] = {};          // lanes of heads whose sum of squares is infinite
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int h = head0 + HEADS * i;
    if (HEADS * (i) + head0 - lane / LANES >= total) break;   // uniform: no head of this pass
    const bool is_q = h < p.Hq;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = bf16_lo(x[i][j]), b = bf16_hi(x[i][j]);
      sum += a * a;
      sum += b * b;
    }
    sum = lanes_sum<LANES>(sum);
    if constexpr (INTERLEAVED) infinite[i] = __ballot(sum == INFINITY);
    const float r = 1.f / sqrtf(sum * (1.f / D) + p.eps);
    const v4u w = is_q ? wq : wk;
    float y[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[2 * j] = bf16_lo(x[i][j]) * r * bf16_lo(w[j]);
      y[2 * j + 1] = bf16_hi(x[i][j]) * r * bf16_hi(w[j]);
    }
    v4u out;
    if constexpr (INTERLEAVED) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        out[j] = pack_bf16(y[2 * j] * c[j] - y[2 * j + 1] * s[j], y[2 * j + 1] * c[j] + y[2 * j] * s[j]);
    } else {
      const v4u wp = is_q ? wq_p : wk_p;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t o = (uint32_t)__shfl((int)x[i][j], partner);
        const float lo = bf16_lo(o) * r * bf16_lo(wp[j]), hi = bf16_hi(o) * r * bf16_hi(wp[j]);
        out[j] = pack_bf16(y[2 * j] * c[2 * j] + lo * s[2 * j], y[2 * j + 1] * c[2 * j + 1] + hi * s[2 * j + 1]);
      }
    }
    if (h < total) put(h, out);
  }
  // Behind the rotated dims an interleaved pair's other value came in times sin 0: NaN
  // where that one is infinite. Those heads' dims again, unrotated: x / infinity. (A
  // half-split pair is there a value and itself.)
  if constexpr (INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      if (infinite[i] == 0) continue;
      const int h = head0 + HEADS * i;
      const v4u w = h < p.Hq ? wq : wk;
      v4u out;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        out[j] = pack_bf16(bf16_lo(x[i][j]) * 0.f * bf16_lo(w[j]), bf16_hi(x[i][j]) * 0.f * bf16_hi(w[j]));
      if (h < total && !turned && (infinite[i] >> lane & 1) != 0) put(h, out);
    }
  }
}

template <int D, bool IL>
hipError_t launch(const QkNormRopeArgs& p, hipStream_t stream) {
  constexpr int HEADS = 64 / (D / 8);
  const int total = p.Hq + p.Hk;
  // one pass a wave while that leaves fewer than 32 waves a CU, two above; past
  // the caches what would not stay in them for its reader (4632 tokens, 64 + 8 heads of
  // 128, inputs that no cache holds: one pass 44.6 us, two 40.4, past the caches 36.4;
  // 1000 tokens, held: one 10.8, two 10.1, past the caches 10.4)
  const int64_t waves1 = p.M * ((total + HEADS - 1) / HEADS), waves2 = p.M * ((total + 2 * HEADS - 1) / (2 * HEADS));
  const bool two = waves1 >= (int64_t)cu_count() * 32;
  const bool past = p.M * total * D * 2 > ((int64_t)32 << 20);
  const int64_t blocks = ((two ? waves2 : waves1) + NORM_WAVES - 1) / NORM_WAVES;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  auto kern = !two ? qk_norm_rope_kernel<D, IL, 1, false> : (past ? qk_norm_rope_kernel<D, IL, 2, true> : qk_norm_rope_kernel<D, IL, 2, false>);
  hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(NORM_WAVES * 64), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_qk_norm_rope(const QkNormRopeArgs& p, int D, bool interleaved, hipStream_t stream) {
  switch (D) {
    case 64: return interleaved ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
    case 128: return interleaved ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
    default: return interleaved ? launch<256, true>(p, stream) : launch<256, false>(p, stream);
  }
}

}  // namespace iqp
