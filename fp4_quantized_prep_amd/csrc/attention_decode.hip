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
  SeqRows r;
  int lo;             // first token that any of its rows sees
  int unit0, units;   // the unit of lo; units up to its end
  int tiles;          // row tiles
  int64_t work;       // tiles * Hk * units
};

template <int ROWS>
__device__ __forceinline__ Seq get_seq(const AttnArgs& p, const SeqRows& r) {
  Seq q;
  q.r = r;
  const int64_t n = r.end - r.begin, rows = n * p.group, held = (int64_t)p.seq.max_blocks << p.seq.log_block;
  const int64_t lo = p.window > 0 ? r.len - n - p.window + 1 : 0, end = r.len < held ? r.len : held;
  q.lo = lo < 0 ? 0 : (int)lo;
  q.unit0 = q.lo / UNIT;
  q.units = end > q.lo ? (int)((end + UNIT - 1) / UNIT) - q.unit0 : 0;
  q.tiles = n > 0 && rows <= p.max_rows ? (int)((rows + ROWS - 1) / ROWS) : 0;
  if (q.tiles > 0 && q.units < 1) q.units = 1;    // rows that see nothing still get their zeros
  q.work = (int64_t)q.tiles * p.Hk * q.units;
  return q;
}

// the running sum of w over the lanes, and its total; in 32 bits where that holds it
__device__ __forceinline__ int64_t scan(int64_t w, int64_t& total) {
  const int lane = threadIdx.x & 63;
  if (__ballot(w >= (1 << 24)) == 0) {
    int v = (int)w;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(v, d);
      if (lane >= d) v += o;
    }
    total = __builtin_amdgcn_readlane(v, 63);
    return v;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t o = __shfl_up((long long)w, d);
    if (lane >= d) w += o;
  }
  total = __shfl((long long)w, 63);
  return w;
}

// a / b of uniform values, a >= 0, b > 0
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// The line of all units, sequence after sequence; within one, row tile by row
// tile, key head by key head. Every wave walks it for itself.
template <int ROWS>
struct Line {
  const AttnArgs& p;
  SeqRows rows64;          // 64 sequences at hand, one a lane
  int64_t sum;             // their units up to the lane's sequence
  int chunk = 0, in_chunk = 0;
  int64_t total = 0;       // units of the whole line
  int64_t base = 0;        // units before sequence q
  Seq q;

  __device__ __forceinline__ explicit Line(const AttnArgs& p_) : p(p_) {
    rows64 = lane_sequence(p.seq, 0);    // kept: most batches have no more
    sum = scan(get_seq<ROWS>(p, rows64).work, total);
    for (int s0 = 64; s0 < p.seq.S; s0 += 64) {
      int64_t t;
      scan(get_seq<ROWS>(p, lane_sequence(p.seq, s0)).work, t);
      total += t;
    }
  }
  // to the sequence that holds unit at (< total); once
  __device__ __forceinline__ void seek(int64_t at) {
    uint64_t past = __ballot(sum > at);
    while (past == 0) {
      base += __shfl((long long)sum, 63);
      chunk += 64;
      rows64 = lane_sequence(p.seq, chunk);
      int64_t t;
      sum = scan(get_seq<ROWS>(p, rows64).work, t);
      past = __ballot(base + sum > at);
    }
    in_chunk = __ffsll((unsigned long long)past) - 1;
    q = get_seq<ROWS>(p, sequence_of_lane(rows64, in_chunk));
    base += __shfl((long long)sum, in_chunk) - q.work;
  }
  // to the sequence that owns row tile slot `item` (as find_sequence finds it); once
  __device__ __forceinline__ void seek_item(int64_t item) {
    constexpr int SHIFT = ROWS == 16 ? 4 : 5;
    int64_t before = 0;
    for (int s0 = 0;; s0 += 64) {
      const int n = __popcll(__ballot(rows64.s < p.seq.S && item_key(rows64, p.group, SHIFT, 1) <= item));
      if (n > 0) {
        q = get_seq<ROWS>(p, sequence_of_lane(rows64, n - 1));
        base = before + __shfl((long long)sum, n - 1) - q.work;
      }
      if (n < 64 || s0 + 64 >= p.seq.S) break;
      int64_t t;
      before += __shfl((long long)sum, 63);
      rows64 = lane_sequence(p.seq, s0 + 64);
      sum = scan(get_seq<ROWS>(p, rows64).work, t);
    }
  }
  // on to the sequence that holds unit at (< total) from one at or before it
  __device__ __forceinline__ void advance(int64_t at) {
    while (at >= base + q.work) {
      base += q.work;
      if (++in_chunk == 64) {
        in_chunk = 0;
        chunk += 64;
        rows64 = lane_sequence(p.seq, chunk);
      }
      q = get_seq<ROWS>(p, sequence_of_lane(rows64, in_chunk));
    }
  }
};

__device__ __forceinline__ int64_t piece_of(int64_t total) {
  // down to a unit: a workgroup that walked several short pairs one after the
  // other would take as long as it saves (19 sequences of up to 71
  // tokens, 8 heads: 20 us with at least four units a workgroup, 10 with one)
  return (total + ATTN_WORKGROUPS - 1) / ATTN_WORKGROUPS;
}

// one workgroup's partial result of a pair: max, sum, output of 16 NT rows
template <int D, int NT>
struct Partial {
  float m[16 * NT], l[16 * NT];
  float o[16 * NT][D];
};

template <int D, int NT>
__global__ __launch_bounds__(DWAVES * 64, 2)
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

  Line<ROWS> line(p);
  if (line.total == 0) return;
  const int64_t per = piece_of(line.total);
  int64_t at = (int64_t)blockIdx.x * per;
  const int64_t stop = at + per < line.total ? at + per : line.total;
  if (at >= stop) return;
  line.seek(at);

  while (at < stop) {
    line.advance(at);
    const Seq& q = line.q;
    const int64_t base = line.base;
    const int s = q.r.s;
    const int64_t q_begin = q.r.begin, q_n = q.r.end - q.r.begin, q_len = q.r.len;
    const int64_t pair = quotient(at - base, q.units);            // row tile and key head of the sequence
    const int64_t off = (at - base) - pair * q.units;
    const int64_t count = q.units - off < stop - at ? q.units - off : stop - at;
    const int64_t tile = quotient(pair, p.Hk);
    const int head = (int)(pair - tile * p.Hk);
    const int64_t row0 = tile * ROWS, rows = q_n * p.group;

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
    for (int64_t u = wave; u < count; u += DWAVES) {
      const int64_t t0 = (q.unit0 + off + u) * UNIT;
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
        const int64_t vhi = held ? q_len - tb : 0, vlo = tile_lo - tb;
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
        uint16_t* dst = p.out + row_offset(q_begin, row0 + r, head, p.group, D, p.ldo) + d;
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

// Joins the pairs whose units went to more than one workgroup. Workgroup (x, z)
// takes every gridDim.y-th row from z on of one pair: the pair that decode
// workgroup x began and did not finish, or (BY_PAIR, where the pairs are fewer
// than the decode workgroups) pair x itself.
template <int D, int NT, bool BY_PAIR>
__global__ __launch_bounds__(JOIN_THREADS)
void attention_join_kernel(AttnArgs p) {
  constexpr int ROWS = 16 * NT;
  __shared__ __attribute__((aligned(16))) JoinSpace<D> lds;
  Line<ROWS> line(p);
  if (line.total == 0) return;                               // no sequence is this kernel's
  const int64_t per = piece_of(line.total);
  const Seq& q = line.q;
  int64_t pair;                                              // of the sequence
  if constexpr (BY_PAIR) {
    const int64_t item = blockIdx.x / (unsigned)p.Hk;
    line.seek_item(item);
    const int64_t tile = item - item_key(q.r, p.group, NT == 1 ? 4 : 5, 1);
    if (tile >= q.tiles) return;
    pair = tile * p.Hk + blockIdx.x % (unsigned)p.Hk;
  } else {
    const int64_t last = (blockIdx.x + (int64_t)1) * per - 1;   // the workgroup's last unit
    if (last >= line.total) return;
    line.seek(last);
    pair = quotient(last - line.base, q.units);
  }
  const int64_t u0 = line.base + pair * q.units, w0 = quotient(u0, per), w1 = quotient(u0 + q.units - 1, per);
  if (w0 == w1 || (!BY_PAIR && w0 != blockIdx.x)) return;    // finished by its workgroup, or begun before this one
  const int64_t tile = quotient(pair, p.Hk), rows = (int64_t)(q.r.end - q.r.begin) * p.group;
  const int head = (int)(pair - tile * p.Hk);
  const Partial<D, NT>* parts = reinterpret_cast<const Partial<D, NT>*>(p.workspace) + 2 * w0;
  const int64_t left = rows - tile * ROWS;
  join_rows<D>(
      lds, blockIdx.y, gridDim.y, left < ROWS ? (int)left : ROWS, (int)(w1 - w0) + 1,
      [&](int i) __attribute__((always_inline)) -> const Partial<D, NT>& { return parts[2 * i + (i == 0 ? 1 : 0)]; },
      [&](int r, int d, float sum, v4f acc) __attribute__((always_inline)) {
        const float inv = inverse_sum(sum);
        uint16_t* dst = p.out + row_offset(q.r.begin, tile * ROWS + r, head, p.group, D, p.ldo) + d;
        *reinterpret_cast<v2u*>(dst) = v2u{pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv)};
      });
}

template <int D, int NT>
hipError_t launch(const AttnArgs& p, hipStream_t stream) {
  hipLaunchKernelGGL((attention_decode_kernel<D, NT>), dim3(ATTN_WORKGROUPS), dim3(DWAVES * 64), 0, stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t pairs = (((p.seq.T * p.group) >> (NT == 1 ? 4 : 5)) + p.seq.S) * p.Hk;   // at most
  if (pairs <= ATTN_WORKGROUPS / 4)
    // each may be in many pieces (8 heads of 131072 tokens: 64 each): a workgroup a row
    hipLaunchKernelGGL((attention_join_kernel<D, NT, true>), dim3((unsigned)pairs, 16 * NT), dim3(JOIN_THREADS), 0, stream, p);
  else
    hipLaunchKernelGGL((attention_join_kernel<D, NT, false>), dim3(ATTN_WORKGROUPS, 2), dim3(JOIN_THREADS), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

int64_t attention_decode_workspace_bytes(int D) {
  return (int64_t)ATTN_WORKGROUPS * 2 * (D == 64 ? sizeof(Partial<64, 2>) : sizeof(Partial<128, 1>));
}

hipError_t launch_attention_decode(const AttnArgs& p, int D, hipStream_t stream) {
  // D 64: two tiles of rows a wave once a sequence brings more than one on average
  // (60 sequences of 8000 tokens, 24 rows a head: 57 us, with one tile 85). D 128
  // leaves no registers for that: one wave a SIMD, half as fast as reading the
  // cache twice (8 sequences of 2000 tokens, 32 rows a head: 33 us against 19).
  if (D == 128) return launch<128, 1>(p, stream);
  return p.seq.T * p.group > 16 * (int64_t)p.seq.S ? launch<64, 2>(p, stream) : launch<64, 1>(p, stream);
}

int64_t attention_workspace_bytes(int D) {
  const int64_t a = attention_decode_workspace_bytes(D), b = attention_prefill_workspace_bytes(D);
  return a > b ? a : b;
}

hipError_t launch_attention(const AttnArgs& args, int D, hipStream_t stream) {
  AttnArgs p = args;
  if (p.seq.T * p.group <= ATTN_DECODE_ROWS * (int64_t)p.seq.S) {
    p.max_rows = (int64_t)1 << 62;
    return launch_attention_decode(p, D, stream);
  }
  // (a single sequence needs one kernel, whatever its number of rows turns out to be)
  const bool alone = p.seq.S == 1 || reach(p) <= ATTN_SHORT_REACH;
  p.max_rows = alone ? 0 : ATTN_DECODE_ROWS;
  const hipError_t e = launch_attention_prefill(p, D, stream);
  if (e != hipSuccess || alone) return e;
  return launch_attention_decode(p, D, stream);
}

}  // namespace iqp
