// Attention of a few query rows per sequence over the FP8 key/value cache.
//
// For a query row at position p of a sequence, over the held tokens t of its
// key head with p - window < t <= p (t <= p without a window):
//   out = sum_t w_t v_t / sum_t w_t,  w_t = exp(scale * q . k_t),
// zeros where no such token exists. k_t and v_t are the cache's codes times
// their block's power of two.
//
// Cache-bound: 2 D bytes a token and key head, read once for all the query
// heads that share it (attention_rows.h). All (sequence, row tile, key head)
// pairs' units of 64 tokens form one line that is cut into equal pieces, one per
// workgroup, whatever the sequences' lengths. A piece covers the end of one pair,
// whole pairs, and the start of another; whole pairs are finished at once, the
// rest go to the workspace as (max, sum, unnormalised output) and a second small
// launch joins them.
//
// Measured, 64 heads of 128 over 8: 64 sequences of 127 to 8191 tokens 111 us,
// 4.75 TB/s; one of 131072 56 us, 4.77 TB/s (a large copy reaches 5.1).
#include "attention_rows.h"

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
  Seq q = {};              // (none: no tiles, no work)

  __device__ __forceinline__ explicit Line(const AttnArgs& p_) : p(p_) {
    rows64 = lane_sequence(p.seq, 0);    // kept: most batches have no more
    sum = scan(get_seq<ROWS>(p, rows64).work, total);
    for (int s0 = 64; s0 < p.seq.S; s0 += 64) {
      int64_t t;
      scan(get_seq<ROWS>(p, lane_sequence(p.seq, s0)).work, t);
      total += t;
    }
  }
  // To the sequence that holds unit at (< total); once. (Should the lengths change
  // under the kernel, which no caller may do, the walks still end: q.work is 0.)
  __device__ __forceinline__ void seek(int64_t at) {
    uint64_t past = __ballot(sum > at);
    while (past == 0) {
      base += __shfl((long long)sum, 63);
      chunk += 64;
      if (chunk >= p.seq.S) {
        in_chunk = 63;
        q.r.s = p.seq.S;
        q.work = 0;
        return;
      }
      rows64 = lane_sequence(p.seq, chunk);
      int64_t t;
      sum = scan(get_seq<ROWS>(p, rows64).work, t);
      past = __ballot(base + sum > at);
    }
    in_chunk = __ffsll((unsigned long long)past) - 1;
    q = get_seq<ROWS>(p, sequence_of_lane(rows64, in_chunk));
    base += __shfl((long long)sum, in_chunk) - q.work;
  }
  // to the sequence that owns row tile slot `item` (as find_sequence finds it; none
  // before the first); once
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
    while (at >= base + q.work && q.r.s < p.seq.S) {
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
__device__ __forceinline__ void decode(const AttnArgs& p, typename FewRows<D, NT, DWAVES>::Lds& lds) {
  constexpr int ROWS = 16 * NT;
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
    if (q.work == 0) return;
    const int64_t base = line.base;
    const int64_t pair = quotient(at - base, q.units);            // row tile and key head of the sequence
    const int64_t off = (at - base) - pair * q.units;
    const int64_t count = q.units - off < stop - at ? q.units - off : stop - at;
    const int64_t tile = quotient(pair, p.Hk);
    const int head = (int)(pair - tile * p.Hk);
    const int64_t row0 = tile * ROWS;
    const bool whole = off == 0 && count == q.units;
    // slot 0: a pair begun by another workgroup; slot 1: one begun here
    Partial<D, NT>* const part = reinterpret_cast<Partial<D, NT>*>(p.workspace) + 2 * (int64_t)blockIdx.x + (off == 0 ? 1 : 0);
    FewRows<D, NT, DWAVES>::run(p, q.r, row0, head, q.unit0 + off, count, lds,
                                [&](int r, int d, float mx, float sum, v4f acc) __attribute__((always_inline)) {
      if (whole) {
        const float inv = inverse_sum(sum);
        uint16_t* dst = p.out + row_offset(q.r.begin, row0 + r, head, p.group, D, p.ldo) + d;
        *reinterpret_cast<v2u*>(dst) = v2u{pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv)};
      } else {
        *reinterpret_cast<v4f*>(&part->o[r][d]) = acc;
        if (d == 0) {
          part->m[r] = mx;
          part->l[r] = sum;
        }
      }
    });
    __syncthreads();
    at += count;
  }
}

template <int D, int NT>
__global__ __launch_bounds__(DWAVES * 64, 2)
void attention_decode_kernel(AttnArgs p) {
  __shared__ __attribute__((aligned(16))) typename FewRows<D, NT, DWAVES>::Lds lds;
  decode<D, NT>(p, lds);
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
    if (tile < 0 || tile >= q.tiles) return;                 // (below 0: offsets that decrease)
    pair = tile * p.Hk + blockIdx.x % (unsigned)p.Hk;
  } else {
    const int64_t last = (blockIdx.x + (int64_t)1) * per - 1;   // the workgroup's last unit
    if (last >= line.total) return;
    line.seek(last);
    if (q.work == 0) return;
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
    // each may be in many pieces (8 heads of 131072 tokens: 64 each): a workgroup a
    // row (that one 50 us, by decode workgroup 57; 512 pairs of up to 8192 tokens 112
    // by decode workgroup, by pair 128)
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
  const int64_t rows = p.seq.T * p.group, S = p.seq.S;
  const bool many = S * p.Hk >= ATTN_MANY_PAIRS || S >= ATTN_MANY;
  const bool direct = rows <= ATTN_DIRECT_ROWS * S && reach(p) <= ATTN_DIRECT_REACH * (many ? 2 : 1);
  if (rows <= ATTN_DECODE_ROWS * S && !direct) {
    p.max_rows = (int64_t)1 << 62;
    return launch_attention_decode(p, D, stream);
  }
  // (a single sequence needs one kernel, whatever its number of rows turns out to be)
  const bool alone = S == 1 || reach(p) <= ATTN_SHORT_REACH;
  p.max_rows = alone ? 0 : ATTN_DECODE_ROWS;
  const hipError_t e = launch_attention_prefill(p, D, stream);
  if (e != hipSuccess || alone) return e;
  return launch_attention_decode(p, D, stream);
}

}  // namespace iqp
