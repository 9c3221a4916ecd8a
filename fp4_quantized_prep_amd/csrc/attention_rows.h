// Attention of up to 16 NT query rows by a workgroup: the formula of
// attention_decode.hip, for the decode kernel and for the prompt kernel's short
// tiles.
//
//   * A wave takes every WAVES-th unit of 64 tokens and loads its 128 D bytes
//     with 16-byte loads straight into MFMA operand registers: a key operand
//     lane holds 16 consecutive dims of a token, a value operand lane 16
//     consecutive tokens of a dim (the cache keeps values that way). Token
//     16 g + 4 c + r of the unit is row 4 g + r of score tile c, so the lane
//     that holds four scores of each tile holds 16 consecutive tokens, and
//     those are its share of the second product's operand: probabilities never
//     leave the lane.
//   * Query rows are the MFMA's columns, NT tiles of 16: the query heads of one
//     key head and their tokens.
//   * The keys widen to bf16 (exact) and meet bf16 queries. The block's key
//     scale multiplies the scores. The values widen to fp16 without their
//     scale (every E4M3 value is one); the probabilities carry it instead:
//     with w'_t = 2^(15 + s_t + e_t - max(s + e)), s in units of log2 and e_t the
//     value exponent, w' <= 2^15 rounds to fp16 (2^-11 relative, an eighth of what
//     bf16 would lose; below 2^-29 of the largest, where fp16 is subnormal,
//     2^-40 of the largest) and sum w = sum w' 2^-e, kept in float32. The power
//     of two leaves with the division.
//   * The waves' results, each relative to its own maximum, meet in LDS.
#pragma once

#include "attention_common.h"

namespace iqp {
namespace {
namespace attn {

template <int D, int NT, int WAVES>
struct FewRows {
  static constexpr int ROWS = 16 * NT;
  static constexpr int KP = D / 64;        // 64-dim groups: two MFMA steps each
  static constexpr int DT = D / 16;        // output tiles

  struct Lds {
    float o[WAVES][ROWS][D + 4];
    float m[WAVES][ROWS], l[WAVES][ROWS];
  };

  // Rows row0 .. of the sequence (at most ROWS), one key head, units u0 .. u0 +
  // count - 1; finish(r, d, max, sum, o) gets dims d .. d + 3 of row row0 + r.
  // All of the workgroup's threads; the caller synchronises before lds is used again.
  template <class Finish>
  static __device__ __forceinline__ void run(const AttnArgs& p, const SeqRows& seq, int64_t row0, int head, int64_t u0, int64_t count,
                                             Lds& lds, const Finish& finish) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int kg = col >> 2;          // 16-token group of the lane's key rows
    const int s = seq.s;
    const int64_t q_begin = seq.begin, q_n = seq.end - seq.begin, q_len = seq.len, rows = q_n * p.group;

    // the queries, and which tokens each column sees: [see_lo, see_hi)
    v8bf fq[NT][2 * KP];
    int64_t see_lo[NT], see_hi[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int64_t r = row0 + 16 * t + col;
      const int64_t rc = r < rows ? r : rows - 1;
      const int64_t i = rc / p.group;
      const uint16_t* src = p.q + (q_begin + i) * p.ldq + ((int64_t)head * p.group + (rc - i * p.group)) * D + 16 * g;
#pragma unroll
      for (int k = 0; k < KP; ++k) {
        fq[t][2 * k] = *reinterpret_cast<const v8bf*>(src + 64 * k);
        fq[t][2 * k + 1] = *reinterpret_cast<const v8bf*>(src + 64 * k + 8);
      }
      const int64_t pos = q_len - q_n + i;
      see_hi[t] = pos + 1;
      see_lo[t] = p.window > 0 && pos + 1 > p.window ? pos + 1 - p.window : 0;
    }
    // every column sees the tokens of [all_lo, all_hi)
    const int64_t i_first = row0 / p.group, i_last = (row0 + ROWS - 1 < rows ? row0 + ROWS - 1 : rows - 1) / p.group;
    const int64_t all_hi = q_len - q_n + i_first + 1;
    const int64_t all_lo = p.window > 0 ? q_len - q_n + i_last + 1 - p.window : 0;
    const int64_t tile_lo = p.window > 0 ? all_hi - p.window : 0;   // no column sees a token before this

    float m[NT], l[NT];
    v4f o[NT][DT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t] = LOWEST;
      l[t] = 0.f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[t][d] = v4f{0.f, 0.f, 0.f, 0.f};
    }

    const int32_t* table = p.seq.table + (int64_t)s * p.seq.ld_table;
    const int lb = p.seq.log_block;
    for (int64_t u = wave; u < count; u += WAVES) {
      const int64_t t0 = (u0 + u) * UNIT;
      // the block of the lane's key rows and the block of its value tokens
      const int64_t bk = (t0 + 16 * kg) >> lb, bv = (t0 + 16 * g) >> lb;
      int64_t pk = bk < p.seq.max_blocks ? table[bk] : -1;
      int64_t pv = bv < p.seq.max_blocks ? table[bv] : -1;
      const bool held = pv >= 0 && pv < p.seq.n_blocks && t0 + 16 * g < q_len;
      pk = pk >= 0 && pk < p.seq.n_blocks ? pk : 0;
      pv = pv >= 0 && pv < p.seq.n_blocks ? pv : 0;
      const int inside = (1 << lb) - 1;
      const uint8_t* kb = p.k_cache + ((pk * p.Hk + head) << lb) * D;
      const uint8_t* vb = p.v_cache + ((pv * p.Hk + head) << lb) * D + ((t0 + 16 * g) & inside);
      v4u kr[4][KP], vr[DT];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint8_t* src = kb + ((t0 + 16 * kg + 4 * c + (col & 3)) & inside) * D + 16 * g;
#pragma unroll
        for (int k = 0; k < KP; ++k) kr[c][k] = *reinterpret_cast<const v4u*>(src + 64 * k);
      }
#pragma unroll
      for (int d = 0; d < DT; ++d) vr[d] = *reinterpret_cast<const v4u*>(vb + ((int64_t)(16 * d + col) << lb));
      const int ke = (int)p.k_scales[pv * p.Hk + head] - 127, ve = (int)p.v_scales[pv * p.Hk + head] - 127;
      const float kmul = p.scale_log2 * pow2(min(max(ke, -126), 127));
      const float ve_f = (float)ve, vinv = pow2(min(max(-ve, -126), 127));

      // scores: tile c, row 4 g + r is token 16 g + 4 c + r
      v4f sc[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[t][c] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int k = 0; k < KP; ++k) {
          const v8bf k0 = widen_bf16(kr[c][k][0], kr[c][k][1]), k1 = widen_bf16(kr[c][k][2], kr[c][k][3]);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            sc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, fq[t][2 * k], sc[t][c], 0, 0, 0);
            sc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, fq[t][2 * k + 1], sc[t][c], 0, 0, 0);
          }
        }
      const bool edge = t0 < all_lo || t0 + UNIT > all_hi || t0 + UNIT > q_len;
      // a block that is not held, or an edge: some token of the unit is out
      if (edge || __ballot(!held) != 0) {
        const int64_t tb = t0 + 16 * g;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int64_t tok = tb + 4 * c + r;
              const bool in = held && tok >= see_lo[t] && tok < see_hi[t];
              sc[t][c][r] = in ? sc[t][c][r] * kmul + ve_f : -INFINITY;
            }
        // whatever lies behind the sequence, before every row's window or in a
        // block that is not held must not reach the product: 0 * NaN
        // (both ends limited on both sides: a window may pass 2^31 tokens)
        const int64_t vhi = held ? q_len - tb : 0, vlo = tile_lo - tb;
        const int hi = vhi > 16 ? 16 : (vhi < 0 ? 0 : (int)vhi), lo = vlo > 16 ? 16 : (vlo < 0 ? 0 : (int)vlo);
#pragma unroll
        for (int d = 0; d < DT; ++d) vr[d] = clear_outside(vr[d], lo, hi);
      } else {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r) sc[t][c][r] = sc[t][c][r] * kmul + ve_f;
      }
      v8h fp[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float mx = sc[t][0][0];
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int r = 0; r < 4; ++r) mx = fmaxf(mx, sc[t][c][r]);
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        // m: the largest score so far less FP16_TOP, or the score itself where that
        // difference would not be exact enough: weights stay within fp16
        float top = mx - FP16_TOP;
        top = mx - top > FP16_TOP ? mx : top;
        const float mn = fmaxf(m[t], top);
        const float alpha = __builtin_amdgcn_exp2f(m[t] - mn);
        m[t] = mn;
        float sum = 0.f;
        float w[16];
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float x = __builtin_amdgcn_exp2f(sc[t][c][r] - mn);
            w[4 * c + r] = x;
            sum += x;
          }
        l[t] = l[t] * alpha + sum * vinv;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int r = 0; r < 4; ++r) o[t][d][r] *= alpha;
#pragma unroll
        for (int c = 0; c < 2; ++c)
          fp[t][c] = v8h{(_Float16)w[8 * c], (_Float16)w[8 * c + 1], (_Float16)w[8 * c + 2], (_Float16)w[8 * c + 3],
                         (_Float16)w[8 * c + 4], (_Float16)w[8 * c + 5], (_Float16)w[8 * c + 6], (_Float16)w[8 * c + 7]};
      }
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const v8h v0 = widen_f16(vr[d][0], vr[d][1]), v1 = widen_f16(vr[d][2], vr[d][3]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          o[t][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, fp[t][0], o[t][d], 0, 0, 0);
          o[t][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, fp[t][1], o[t][d], 0, 0, 0);
        }
      }
    }

    // join the waves: each puts its rows, relative to its own maximum, into LDS
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float sum = l[t];
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (g == 0) {
        lds.m[wave][16 * t + col] = m[t];
        lds.l[wave][16 * t + col] = sum;
      }
#pragma unroll
      for (int d = 0; d < DT; ++d) *reinterpret_cast<v4f*>(&lds.o[wave][16 * t + col][16 * d + 4 * g]) = o[t][d];
    }
    __syncthreads();
    for (int i = tid; i < ROWS * (D / 4); i += WAVES * 64) {
      const int r = i / (D / 4), d = 4 * (i % (D / 4));
      if (row0 + r >= rows) break;
      float mx = lds.m[0][r];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) mx = fmaxf(mx, lds.m[w][r]);
      float sum = 0.f;
      v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const float a = __builtin_amdgcn_exp2f(lds.m[w][r] - mx);
        sum += lds.l[w][r] * a;
        const v4f x = *reinterpret_cast<const v4f*>(&lds.o[w][r][d]);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] += x[j] * a;
      }
      finish(r, d, mx, sum, acc);
    }
  }
};

}  // namespace attn
}  // namespace
}  // namespace iqp
