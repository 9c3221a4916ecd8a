// Attention of a few query rows per sequence over the FP8 key/value cache.
//
// For a query row at position p of a sequence, over the held tokens t of its
// key head with p - window < t <= p (t <= p without a window):
//   out = sum_t w_t v_t / sum_t w_t,  w_t = exp(scale * q . k_t),
// zeros where no such token exists. k_t and v_t are the cache's codes times
// their block's power of two.
//
// Cache-bound: 2 D bytes a token and key head, read once for all the query
// heads that share it. What the layout does about it:
//   * the cache is cut into units of 64 tokens. A wave loads a unit's 128 D
//     bytes with 16-byte loads straight into MFMA operand registers: a key
//     operand lane holds 16 consecutive dims of a token, a value operand lane
//     16 consecutive tokens of a dim (the cache keeps values that way). Token
//     16 g + 4 c + r of the unit is row 4 g + r of score tile c, so the lane
//     that holds four scores of each tile holds 16 consecutive tokens, and
//     those are its share of the second product's operand: probabilities never
//     leave the lane.
//   * query rows are the MFMA's columns, NT tiles of 16: the query heads of
//     one key head and their tokens.
//   * the keys widen to bf16 (exact) and meet bf16 queries. The block's key
//     scale multiplies the scores. The values widen to fp16 without their
//     scale (every E4M3 value is one); the probabilities carry it instead:
//     with w'_t = 2^(s_t + e_t - max(s + e)), s in units of log2 and e_t the
//     value exponent, w' <= 1 rounds to fp16 (2^-11 relative, half of what
//     bf16 would lose) and sum w = sum w' 2^-e, kept in float32.
//   * all (sequence, row tile, key head) pairs' units form one line that is cut
//     into equal pieces, one per workgroup, whatever the sequences' lengths.
//     A piece covers the end of one pair, whole pairs, and the start of
//     another; whole pairs are finished at once, the rest go to the workspace as
//     (max, sum, unnormalised output) and a second small launch joins them.
#include "attention_common.h"

namespace iqp {
namespace {

using namespace attn;

constexpr int DWAVES = 4;

// What a workgroup needs of a sequence.
struct Seq {
  int64_t begin;      // its first row in the batch
  int64_t n;          // its rows (tokens)
  int64_t len;        // tokens held, those rows included
  int64_t lo;         // first token that any of its rows sees
  int64_t unit0;      // the unit of lo
  int64_t units;      // units up to len
  int64_t tiles;      // row tiles
  int64_t work;       // tiles * Hk * units
};

template <int ROWS>
__device__ __forceinline__ Seq get_seq(const AttnArgs& p, int s) {
  Seq q;
  q.begin = seq_begin(p.seq, s);
  q.n = seq_begin(p.seq, s + 1) - q.begin;
  q.len = p.seq.lens[s];
  const int64_t held = (int64_t)p.seq.max_blocks << p.seq.log_block;
  const int64_t rows = q.n * p.group;
  q.lo = 0;
  if (p.window > 0) {
    q.lo = q.len - q.n - p.window + 1;
    if (q.lo < 0) q.lo = 0;
  }
  const int64_t end = q.len < held ? q.len : held;
  q.unit0 = q.lo / UNIT;
  q.units = end > q.lo ? (end + UNIT - 1) / UNIT - q.unit0 : 0;
  q.tiles = q.n > 0 && rows <= p.max_rows ? (rows + ROWS - 1) / ROWS : 0;
  if (q.tiles > 0 && q.units < 1) q.units = 1;    // rows that see nothing still get their zeros
  q.work = q.tiles * p.Hk * q.units;
  return q;
}

// total work, and the sequence and offset that unit `at` falls in (s = S: past
// the end). Every wave computes it for itself, 64 sequences at a time.
template <int ROWS>
__device__ __forceinline__ int64_t locate(const AttnArgs& p, int64_t at, int& s_out, int64_t& base_out) {
  const int lane = threadIdx.x & 63;
  int64_t total = 0;
  s_out = p.seq.S;
  base_out = 0;
  for (int s0 = 0; s0 < p.seq.S; s0 += 64) {
    const int64_t w = s0 + lane < p.seq.S ? get_seq<ROWS>(p, s0 + lane).work : 0;
    int64_t sum = w;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t o = __shfl_up((long long)sum, d);
      if (lane >= d) sum += o;
    }
    const uint64_t past = __ballot(total + sum > at && w > 0);
    if (past != 0 && s_out == p.seq.S) {
      const int f = __ffsll((unsigned long long)past) - 1;
      s_out = s0 + f;
      base_out = total + __shfl((long long)(sum - w), f);
    }
    total += __shfl((long long)sum, 63);
  }
  return total;
}

__device__ __forceinline__ int64_t piece_of(const AttnArgs& p, int64_t total) {
  const int64_t per = (total + ATTN_WORKGROUPS - 1) / ATTN_WORKGROUPS;
  return per < DWAVES ? DWAVES : per;     // at least a unit a wave
}

// one workgroup's partial result of a pair: max, sum, output of 16 NT rows
template <int D, int NT>
struct Partial {
  float m[16 * NT], l[16 * NT];
  float o[16 * NT][D];
};

template <int D, int NT>
__global__ __launch_bounds__(DWAVES * 64)
void attention_decode_kernel(AttnArgs p) {
  constexpr int ROWS = 16 * NT;
  constexpr int KP = D / 64;        // 64-dim groups: two MFMA steps each
  constexpr int DT = D / 16;        // output tiles
  __shared__ __attribute__((aligned(16))) float lds_o[DWAVES][ROWS][D + 4];
  __shared__ float lds_m[DWAVES][ROWS], lds_l[DWAVES][ROWS];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int kg = col >> 2;          // 16-token group of the lane's key rows

  int s;
  int64_t base;
  // (the total does not depend on the position asked for)
  int s_first;
  int64_t base_first;
  const int64_t total = locate<ROWS>(p, 0, s_first, base_first);
  const int64_t per = piece_of(p, total);
  int64_t at = (int64_t)blockIdx.x * per;
  const int64_t stop = at + per < total ? at + per : total;
  if (at >= stop) return;
  locate<ROWS>(p, at, s, base);
  Seq q = get_seq<ROWS>(p, s);

  while (at < stop) {
    while (at >= base + q.work) {   // on to the next sequence with work
      base += q.work;
      q = get_seq<ROWS>(p, ++s);
    }
    const int64_t pair = (at - base) / q.units;              // row tile and key head of the sequence
    const int64_t off = (at - base) - pair * q.units;
    const int64_t count = q.units - off < stop - at ? q.units - off : stop - at;
    const int64_t tile = pair / p.Hk;
    const int head = (int)(pair - tile * p.Hk);
    const int64_t row0 = tile * ROWS, rows = q.n * p.group;

    // the queries, and which tokens each column sees: [see_lo, see_hi)
    v8bf fq[NT][2 * KP];
    int64_t see_lo[NT], see_hi[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int64_t r = row0 + 16 * t + col;
      const int64_t rc = r < rows ? r : rows - 1;
      const int64_t i = rc / p.group;
      const uint16_t* src = p.q + (q.begin + i) * p.ldq + ((int64_t)head * p.group + (rc - i * p.group)) * D + 16 * g;
#pragma unroll
      for (int k = 0; k < KP; ++k) {
        fq[t][2 * k] = *reinterpret_cast<const v8bf*>(src + 64 * k);
        fq[t][2 * k + 1] = *reinterpret_cast<const v8bf*>(src + 64 * k + 8);
      }
      const int64_t pos = q.len - q.n + i;
      see_hi[t] = pos + 1;
      see_lo[t] = p.window > 0 && pos + 1 > p.window ? pos + 1 - p.window : 0;
    }
    // every column sees the tokens of [all_lo, all_hi)
    const int64_t i_first = row0 / p.group, i_last = (row0 + ROWS - 1 < rows ? row0 + ROWS - 1 : rows - 1) / p.group;
    const int64_t all_hi = q.len - q.n + i_first + 1;
    const int64_t all_lo = p.window > 0 ? q.len - q.n + i_last + 1 - p.window : 0;
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
    for (int64_t u = wave; u < count; u += DWAVES) {
      const int64_t t0 = (q.unit0 + off + u) * UNIT;
      // the block of the lane's key rows and the block of its value tokens
      const int64_t bk = (t0 + 16 * kg) >> lb, bv = (t0 + 16 * g) >> lb;
      int64_t pk = bk < p.seq.max_blocks ? table[bk] : -1;
      int64_t pv = bv < p.seq.max_blocks ? table[bv] : -1;
      const bool held = pv >= 0 && pv < p.seq.n_blocks && t0 + 16 * g < q.len;
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
      const bool edge = t0 < all_lo || t0 + UNIT > all_hi || t0 + UNIT > q.len;
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
        const int64_t vhi = held ? q.len - tb : 0, vlo = tile_lo - tb;
        const int hi = vhi > 16 ? 16 : (int)vhi, lo = vlo > 16 ? 16 : (int)vlo;
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
        const float mn = fmaxf(m[t], mx);
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

    // join the four waves: each puts its rows, relative to its own maximum,
    // into LDS
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float sum = l[t];
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (g == 0) {
        lds_m[wave][16 * t + col] = m[t];
        lds_l[wave][16 * t + col] = sum;
      }
#pragma unroll
      for (int d = 0; d < DT; ++d) *reinterpret_cast<v4f*>(&lds_o[wave][16 * t + col][16 * d + 4 * g]) = o[t][d];
    }
    __syncthreads();
    const bool whole = off == 0 && count == q.units;
    Partial<D, NT>* part = nullptr;
    if (!whole) {
      // slot 0: a pair begun by another workgroup; slot 1: one begun here
      part = reinterpret_cast<Partial<D, NT>*>(p.workspace) + 2 * (int64_t)blockIdx.x + (off == 0 ? 1 : 0);
    }
    for (int i = tid; i < ROWS * (D / 4); i += DWAVES * 64) {
      const int r = i / (D / 4), d = 4 * (i % (D / 4));
      if (row0 + r >= rows) break;
      float mx = lds_m[0][r];
#pragma unroll
      for (int w = 1; w < DWAVES; ++w) mx = fmaxf(mx, lds_m[w][r]);
      float sum = 0.f;
      v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < DWAVES; ++w) {
        const float a = __builtin_amdgcn_exp2f(lds_m[w][r] - mx);
        sum += lds_l[w][r] * a;
        const v4f x = *reinterpret_cast<const v4f*>(&lds_o[w][r][d]);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] += x[j] * a;
      }
      if (whole) {
        const float inv = inverse_sum(sum);
        const int64_t tok = (row0 + r) / p.group;
        uint16_t* dst = p.out + (q.begin + tok) * p.ldo + ((int64_t)head * p.group + (row0 + r - tok * p.group)) * D + d;
        *reinterpret_cast<v2u*>(dst) = v2u{pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv)};
      } else {
        *reinterpret_cast<v4f*>(&part->o[r][d]) = acc;
        if (d == 0) {
          part->m[r] = mx;
          part->l[r] = sum;
        }
      }
    }
    __syncthreads();
    at += count;
  }
}

// Joins the pairs whose units went to more than one workgroup. A workgroup per
// item = row tile (in the numbering of find_sequence) and key head.
template <int D, int NT>
__global__ __launch_bounds__(256)
void attention_join_kernel(AttnArgs p) {
  constexpr int ROWS = 16 * NT;
  const int tid = threadIdx.x;
  int s_first;
  int64_t base_first;
  const int64_t total = locate<ROWS>(p, 0, s_first, base_first);
  const int64_t per = piece_of(p, total);
  const int64_t pair_item = blockIdx.x;                      // row tile slot
  const int s = find_sequence(p.seq, pair_item, p.group, NT == 1 ? 4 : 5, 1);
  const int64_t tile = pair_item - item_key(p.seq, s, p.group, NT == 1 ? 4 : 5, 1);
  const Seq q = get_seq<ROWS>(p, s);
  if (tile >= q.tiles) return;
  // where the sequence's work begins
  int64_t base = 0;
  const int lane = tid & 63;
  for (int s0 = 0; s0 < s; s0 += 64) {
    int64_t w = s0 + lane < s ? get_seq<ROWS>(p, s0 + lane).work : 0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) w += __shfl_xor((long long)w, d);
    base += w;
  }
  const int head = blockIdx.y;
  const int64_t u0 = base + (tile * p.Hk + head) * q.units, u1 = u0 + q.units;
  const int64_t w0 = u0 / per, w1 = (u1 - 1) / per;
  if (w0 == w1) return;                                      // finished by its workgroup
  const int64_t row0 = tile * ROWS, rows = q.n * p.group;
  const Partial<D, NT>* parts = reinterpret_cast<const Partial<D, NT>*>(p.workspace);
  for (int i = tid; i < ROWS * (D / 4); i += 256) {
    const int r = i / (D / 4), d = 4 * (i % (D / 4));
    if (row0 + r >= rows) break;
    float mx = LOWEST;
    for (int64_t w = w0; w <= w1; ++w) mx = fmaxf(mx, parts[2 * w + (w == w0 ? 1 : 0)].m[r]);
    float sum = 0.f;
    v4f acc = {0.f, 0.f, 0.f, 0.f};
    for (int64_t w = w0; w <= w1; ++w) {
      const Partial<D, NT>& x = parts[2 * w + (w == w0 ? 1 : 0)];
      const float a = __builtin_amdgcn_exp2f(x.m[r] - mx);
      sum += x.l[r] * a;
      const v4f v = *reinterpret_cast<const v4f*>(&x.o[r][d]);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] += v[j] * a;
    }
    const float inv = inverse_sum(sum);
    const int64_t tok = (row0 + r) / p.group;
    uint16_t* dst = p.out + (q.begin + tok) * p.ldo + ((int64_t)head * p.group + (row0 + r - tok * p.group)) * D + d;
    *reinterpret_cast<v2u*>(dst) = v2u{pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv)};
  }
}

template <int D, int NT>
hipError_t launch(const AttnArgs& p, hipStream_t stream) {
  const int64_t tiles = ((p.seq.T * p.group) >> (NT == 1 ? 4 : 5)) + p.seq.S;   // row tiles, at most
  if (tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL((attention_decode_kernel<D, NT>), dim3(ATTN_WORKGROUPS), dim3(DWAVES * 64), 0, stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attention_join_kernel<D, NT>), dim3((unsigned)tiles, (unsigned)p.Hk), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

int64_t attention_decode_workspace_bytes(int D) {
  return (int64_t)ATTN_WORKGROUPS * 2 * (D == 64 ? sizeof(Partial<64, 2>) : sizeof(Partial<128, 2>));
}

hipError_t launch_attention_decode(const AttnArgs& p, int D, hipStream_t stream) {
  // two tiles of rows a wave once a sequence brings more than one on average
  const bool two = p.seq.T * p.group > 16 * (int64_t)p.seq.S;
  if (D == 64) return two ? launch<64, 2>(p, stream) : launch<64, 1>(p, stream);
  return two ? launch<128, 2>(p, stream) : launch<128, 1>(p, stream);
}

int64_t attention_workspace_bytes(int D) {
  const int64_t a = attention_decode_workspace_bytes(D), b = attention_prefill_workspace_bytes(D);
  return a > b ? a : b;
}

hipError_t launch_attention(const AttnArgs& args, int D, hipStream_t stream) {
  AttnArgs p = args;
  if (p.seq.T <= ATTN_DECODE_TOKENS * (int64_t)p.seq.S) {
    p.max_rows = (int64_t)1 << 62;
    return launch_attention_decode(p, D, stream);
  }
  // a single sequence needs one kernel, whatever its number of rows turns out to be
  p.max_rows = p.seq.S == 1 ? 0 : ATTN_DECODE_ROWS;
  const hipError_t e = launch_attention_prefill(p, D, stream);
  if (e != hipSuccess || p.seq.S == 1) return e;
  return launch_attention_decode(p, D, stream);
}

}  // namespace iqp
