// Around the products by expert: the router's choice of experts, the entries of
// a batch sorted by group, and every token's weighted sum of its experts' rows.
#include <type_traits>

#include "iqprep.h"
#include "layer_common.h"
#include "row_groups.h"

namespace iqp {
namespace {

// ---------------------------------------------------------------- the router

// A choice and its expert as an unsigned integer of the order that the experts are
// taken in: the order of float64, NaN above all, zeros of either sign alike, with
// the index, counted down, in place of the last ten bits. A logit (float32 at
// most) keeps all of its bits; a sum of score and bias keeps 42 of its mantissa,
// eight fewer than its score is good to. Never 0.
__device__ __forceinline__ uint64_t key_of(double v, int e) {
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  const uint64_t k = v != v ? ~0ull : b >> 63 ? ~b : b | 1ull << 63;
  return (k & ~1023ull) | (uint64_t)(1023 - e);
}

__device__ __forceinline__ int expert_of(uint64_t key) { return 1023 - (int)(key & 1023); }

template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
  return o > v ? o : v;
}

// the largest of a token's lanes (a row of 16, or all), in each of them
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  if constexpr (LANES == 16) {
    v = dpp_max<0xB1>(v);      // lane ^ 1, ^ 2, mirrored in 8, in 16
    v = dpp_max<0x4E>(v);
    v = dpp_max<0x141>(v);
    return dpp_max<0x140>(v);
  } else {
    v = dpp_max<0x111>(v);     // shifted by 1, 2, 4, 8, row to row, half to half
    v = dpp_max<0x112>(v);
    v = dpp_max<0x114>(v);
    v = dpp_max<0x118>(v);
    v = dpp_max<0x142, 0xA>(v);
    v = dpp_max<0x143, 0xC>(v);
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
  }
}

// of 64 bits: the upper halves, then the lower ones of the lanes that have the largest
template <int LANES>
__device__ __forceinline__ uint64_t lanes_max(uint64_t v) {
  const uint32_t hi = lanes_max<LANES>((uint32_t)(v >> 32));
  return (uint64_t)hi << 32 | lanes_max<LANES>((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
}

template <int LANES>
__device__ __forceinline__ double lanes_sum(double v) {
#pragma unroll
  for (int m = LANES / 2; m; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

__device__ __forceinline__ double score_of(double z, int scoring) {
  if (scoring == IQP_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-z));
  return sqrt((z > 0.0 ? z : 0.0) + log1p(exp(-fabs(z))));    // sqrt of softplus
}

// 1 / (1 + e^-z) for |z| < 690 to 2^-50 of itself, in half of the instructions that
// exp and a division take: e^-z = 2^n e^r with r within ln 2 / 2 of 0, e^r by its
// series (the next term is below 2^-52), the reciprocal by two Newton steps.
__device__ __forceinline__ double sigmoid_of(double z) {
  const double n = __builtin_rint(z * -1.4426950408889634);      // 1 / ln 2
  double r = __builtin_fma(n, -0.6931471805599453, -z);          // ln 2, and what it lacks
  r = __builtin_fma(n, -2.3190468138462996e-17, r);
  constexpr double OVER_FACTORIAL[] = {1.0 / 479001600, 1.0 / 39916800, 1.0 / 3628800, 1.0 / 362880, 1.0 / 40320, 1.0 / 5040,
                                       1.0 / 720, 1.0 / 120, 1.0 / 24, 1.0 / 6, 1.0 / 2, 1.0, 1.0};      // 12! .. 0!
  double e = OVER_FACTORIAL[0];
#pragma unroll
  for (int k = 1; k < 13; ++k) e = __builtin_fma(e, r, OVER_FACTORIAL[k]);
  const double d = 1.0 + __builtin_ldexp(e, (int)n);
  double q = __builtin_amdgcn_rcp(d);
  q = __builtin_fma(__builtin_fma(-d, q, 1.0), q, q);
  return __builtin_fma(__builtin_fma(-d, q, 1.0), q, q);
}

// LANES lanes a token, expert LANES v + lane its lane's v-th value. Scores and
// choices are float64, so that which expert is taken does not hang on how an
// exponential is rounded. Bound by its instructions: 256 experts, top 8, with a bias:
// 4.1 us for a token (2.5 of it a launch), 7.6 to 8.5 for 4632 (2 of it the scores, 2.5 the
// choice), whose logits' read takes 1; 1024 experts 10.7 and 25.
template <int LANES, int VPL>
__global__ __launch_bounds__(256)
void moe_route_kernel(MoeRouteArgs p) {
  const int lane = threadIdx.x & (LANES - 1);
  const int64_t m = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LANES;
  if (m >= p.M) return;
  const float NONE = -__builtin_inff();
  // every load before anything waits: expert LANES v + lane, or the first one again
  float z[VPL], b[VPL] = {};
  if (p.half) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int e = LANES * v + lane;
      z[v] = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p.logits)[m * p.ld + (e < p.E ? e : 0)] << 16);
    }
  } else {
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int e = LANES * v + lane;
      z[v] = reinterpret_cast<const float*>(p.logits)[m * p.ld + (e < p.E ? e : 0)];
    }
  }
  if (p.bias) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) b[v] = p.bias[LANES * v + lane < p.E ? LANES * v + lane : 0];
  }
#pragma unroll
  for (int v = 0; v < VPL; ++v) z[v] = LANES * v + lane < p.E ? z[v] : NONE;
  double top = 0.0, sum = 1.0;     // of softmax over all experts, where that is asked for
  if (p.scoring == IQP_SCORE_SOFTMAX && (p.bias || !p.renormalize)) {
    float t = NONE;
#pragma unroll
    for (int v = 0; v < VPL; ++v) t = z[v] > t ? z[v] : t;
#pragma unroll
    for (int d = LANES / 2; d; d >>= 1) {
      const float o = __shfl_xor(t, d);
      t = o > t ? o : t;
    }
    top = (double)t;
    sum = 0.0;
#pragma unroll
    for (int v = 0; v < VPL; ++v) sum += z[v] == NONE ? 0.0 : exp((double)z[v] - top);
    sum = lanes_sum<LANES>(sum);
  }
  // a NaN among the logits, or +inf, makes every softmax NaN: the logits decide then
  const bool no_scores = sum != sum;
  uint64_t key[VPL];
  double score[VPL];       // with a bias: of every expert, as the choice goes by it
  const auto slow = [&](int v) __attribute__((always_inline)) {
    return p.scoring == IQP_SCORE_SOFTMAX ? exp((double)z[v] - top) / sum : score_of((double)z[v], p.scoring);
  };
  // Few sigmoids a lane by few instructions (us, so / by exp and a division: 1024
  // tokens, top 8, 256 experts (4 a lane) 4.9 / 5.2, 64 (1) 3.3 / 3.8; 16384 of 16 (1) 3.3 /
  // 4.8, but of 256 (16 a lane) 23.4 / 20.1).
  // Which of the two a value takes goes by the value alone, so that a token's scores
  // do not hang on the tokens beside it in the wave.
  constexpr bool FEW = VPL <= 4;
  if (FEW && p.bias) {
    if (p.scoring == IQP_SCORE_SIGMOID) {
      bool far[VPL], any = false;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        far[v] = !(fabsf(z[v]) < 690.f || z[v] == NONE);
        any = any || far[v];
        score[v] = sigmoid_of((double)z[v]);
      }
      if (__ballot(any)) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) score[v] = far[v] ? slow(v) : score[v];
      }
    } else {
#pragma unroll
      for (int v = 0; v < VPL; ++v) score[v] = slow(v);
    }
  }
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int e = LANES * v + lane;
    double c = (double)z[v];
    if (p.bias) {
      score[v] = z[v] == NONE ? 0.0 : FEW ? score[v] : slow(v);
      c = z[v] == NONE || no_scores ? c : score[v] + (double)b[v];
    }
    key[v] = e < p.E ? key_of(c, e) : 0;
  }
  int mine = 0;      // lane j: the j-th choice
  if constexpr (LANES == 64) {
    // Upper halves alone, where one expert has the largest, as it nearly always
    // is but for bf16 logits; else the lower ones of those that share it. (4632 tokens,
    // top 8, without a bias, this way / whole keys throughout and a load after the other:
    // 256 experts 6.6 / 7.1 us, bf16 6.8; 1024 experts 17.0 / 54.9.)
    uint32_t hi[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) hi[v] = (uint32_t)(key[v] >> 32);
    for (int j = 0; j < p.top; ++j) {
      uint32_t best = hi[0];
#pragma unroll
      for (int v = 1; v < VPL; ++v) best = hi[v] > best ? hi[v] : best;
      best = lanes_max<LANES>(best);
      int n = 0, e = 0;
#pragma unroll
      for (int v = 0; v < VPL; ++v) n += __popcll(__ballot(hi[v] == best));
      const auto take = [&](int v, bool is) __attribute__((always_inline)) {
        const uint64_t at = __ballot(is);
        e = at ? LANES * v + __builtin_ctzll(at) : e;
        hi[v] = is ? 0 : hi[v];
      };
      if (n == 1) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) take(v, hi[v] == best);
      } else {
        uint32_t low = 0;
#pragma unroll
        for (int v = 0; v < VPL; ++v) low = hi[v] == best && (uint32_t)key[v] > low ? (uint32_t)key[v] : low;
        low = lanes_max<LANES>(low);
#pragma unroll
        for (int v = 0; v < VPL; ++v) take(v, hi[v] == best && (uint32_t)key[v] == low);
      }
      mine = lane == j ? e : mine;
    }
  } else {
    for (int j = 0; j < p.top; ++j) {
      uint64_t best = key[0];
#pragma unroll
      for (int v = 1; v < VPL; ++v) best = key[v] > best ? key[v] : best;
      best = lanes_max<LANES>(best);
#pragma unroll
      for (int v = 0; v < VPL; ++v) key[v] = key[v] == best ? 0 : key[v];
      mine = lane == j ? expert_of(best) : mine;
    }
  }
  // what the chosen experts' lanes hold
  double w = 0.0;
  if (p.bias) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const double o = __shfl(score[v], mine % LANES, LANES);
      w = mine / LANES == v ? o : w;
    }
  } else {
    float x = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const float o = __shfl(z[v], mine % LANES, LANES);
      x = mine / LANES == v ? o : x;
    }
    if (p.scoring != IQP_SCORE_SOFTMAX) w = score_of((double)x, p.scoring);
    else if (!p.renormalize) w = x == NONE ? 0.0 : exp((double)x - top) / sum;
    else w = x == NONE ? 0.0 : exp((double)x - (double)__shfl(x, 0, LANES));   // relative to the largest chosen one alone
  }
  w = lane < p.top ? w : 0.0;
  if (p.renormalize) {
    const double total = lanes_sum<LANES>(w);
    w = total == 0.0 ? 0.0 : w / total;
  }
  if (lane < p.top) {
    p.weights[m * p.top + lane] = (float)(w * (double)p.scale);
    p.experts[m * p.top + lane] = mine;
  }
}

// ------------------------------------------------------- rows sorted by group

constexpr int SORT_THREADS = 1024, SORT_WAVES = SORT_THREADS / 64;

__device__ __forceinline__ int group_of(const GroupRowsArgs& p, int64_t i) {
  const int g = p.index[i];
  return g >= 0 && g < p.G ? g : p.G;
}

// entries of each group in chunk blockIdx.x
__global__ __launch_bounds__(SORT_THREADS)
void group_count_kernel(GroupRowsArgs p) {
  __shared__ int count[MAX_GROUPS];
  for (int g = threadIdx.x; g < p.G; g += SORT_THREADS) count[g] = 0;
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * p.chunk, end = first + p.chunk < p.R ? first + p.chunk : p.R;
  for (int64_t i = first + threadIdx.x; i < end; i += SORT_THREADS) {
    const int g = group_of(p, i);
    if (g < p.G) atomicAdd(&count[g], 1);
  }
  __syncthreads();
  for (int g = threadIdx.x; g < p.G; g += SORT_THREADS) p.counts[(int64_t)blockIdx.x * p.G + g] = count[g];
}

// Stable: an entry's place is the number of entries of lower groups, of its group
// in chunks and waves before its own (the integer atomics add in any order), and
// of its group before it in its wave (found by comparing the bits of the 64 lanes'
// groups). Bound by its few dependent steps: 8 entries 3.1 us, 2048 of 256 groups 4.2,
// 37056 7.4 with the counts' launch, for 1.2 MB.
__global__ __launch_bounds__(SORT_THREADS)
void group_place_kernel(GroupRowsArgs p) {
  __shared__ int at[SORT_WAVES * MAX_GROUPS];
  __shared__ int counted[2 * MAX_GROUPS];
  __shared__ int sums[SORT_WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t first = (int64_t)blockIdx.x * p.chunk, end = first + p.chunk < p.R ? first + p.chunk : p.R;
  const int64_t share = ((p.chunk + SORT_THREADS - 1) / SORT_THREADS) * 64;      // entries of a wave
  const int64_t mine = first + wave * share, mine_end = mine + share < end ? mine + share : end;
  // the wave's first entries (all that it has, up to 2^17 in all) and the counts are
  // asked for before anything waits
  const int own = mine + lane < mine_end ? group_of(p, mine + lane) : p.G;
  // Entries of a group before this chunk, and from it on: the chunks' counts, shared out
  // to as many threads a group as there are, as many loads at a time as each has chunks
  // (all chunks by one thread, 16 at a time / so: 37056 entries of 256 groups 7.8 / 7.4 us,
  // of 64 7.2 / 6.3, 131072 of 256 11.3 / 9.5); or, where no launch has counted, entry by
  // entry below.
  int earlier = 0, later = 0;
  const int wide = p.G > 64 ? 32 - __builtin_clz(p.G - 1) : 6, mate = tid >> wide, mine_g = tid & ((1 << wide) - 1);
  const auto add_counts = [&](auto at_once) __attribute__((always_inline)) {
    constexpr int LOADS = decltype(at_once)::value;
    for (int c0 = mate; c0 < (int)gridDim.x; c0 += LOADS * SORT_THREADS >> wide) {
      int n[LOADS];
#pragma unroll
      for (int k = 0; k < LOADS; ++k) {
        const int c = c0 + (k * SORT_THREADS >> wide);
        n[k] = p.counts[(int64_t)(c < (int)gridDim.x ? c : 0) * p.G + mine_g];
      }
#pragma unroll
      for (int k = 0; k < LOADS; ++k) {
        const int c = c0 + (k * SORT_THREADS >> wide);
        earlier += c < (int)blockIdx.x ? n[k] : 0;
        later += c >= (int)blockIdx.x && c < (int)gridDim.x ? n[k] : 0;
      }
    }
  };
  if (p.counts && mine_g < p.G) {
    const int each = (int)((gridDim.x + (SORT_THREADS >> wide) - 1) / (unsigned)(SORT_THREADS >> wide));
    if (each <= 4) add_counts(std::integral_constant<int, 4>());
    else if (each <= 12) add_counts(std::integral_constant<int, 12>());
    else add_counts(std::integral_constant<int, 16>());
  }
  const bool several = gridDim.x > 1, count_all = !p.counts && several;
  for (int g = tid; g < SORT_WAVES * p.G; g += SORT_THREADS) at[g] = 0;
  if (several)
    for (int g = tid; g < p.G; g += SORT_THREADS) counted[g] = counted[MAX_GROUPS + g] = 0;
  __syncthreads();
  if (own < p.G) atomicAdd(&at[wave * p.G + own], 1);
  for (int64_t i = mine + 64 + lane; i < mine_end; i += 64) {
    const int g = group_of(p, i);
    if (g < p.G) atomicAdd(&at[wave * p.G + g], 1);
  }
  if (p.counts && mine_g < p.G) {
    atomicAdd(&counted[mine_g], earlier);
    atomicAdd(&counted[MAX_GROUPS + mine_g], later);
  }
  if (count_all)
    for (int64_t i = tid; i < p.R; i += SORT_THREADS) {      // (eight loads at a time: 2048 entries 5.0 us for 4.2, 8192 5.3 for 5.4)
      const int g = group_of(p, i);
      if (g < p.G) atomicAdd(&counted[i < first ? g : MAX_GROUPS + g], 1);
    }
  __syncthreads();
  int before = 0, all = 0;      // thread g: its group's
  if (tid < p.G) {
    if (several) {
      before = counted[tid];
      all = before + counted[MAX_GROUPS + tid];
    } else {
#pragma unroll
      for (int w = 0; w < SORT_WAVES; ++w) all += at[w * p.G + tid];
    }
  }
  const int upto = groups::wave_scan(all);
  if (lane == 63) sums[wave] = upto;
  __syncthreads();
  int start = upto - all, total = 0;
#pragma unroll
  for (int w = 0; w < SORT_WAVES; ++w) {
    start += w < wave ? sums[w] : 0;
    total += sums[w];
  }
  if (tid < p.G) {
    if (blockIdx.x == 0) p.offsets[tid] = start;
    int to = start + before;
#pragma unroll
    for (int w = 0; w < SORT_WAVES; ++w) {
      const int n = at[w * p.G + tid];
      at[w * p.G + tid] = to;
      to += n;
    }
  }
  if (blockIdx.x == 0 && tid == 0) p.offsets[p.G] = total;
  __syncthreads();
  const int bits = 32 - __builtin_clz(p.G);      // of 0 .. G
  for (int64_t i0 = mine; i0 < mine_end; i0 += 64) {
    const int64_t i = i0 + lane;
    const int g = i0 == mine ? own : i < mine_end ? group_of(p, i) : p.G;
    uint64_t same = ~0ull;
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot(g >> b & 1);
      same &= g >> b & 1 ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    int to = -1;
    if (g < p.G) {
      const int base = at[wave * p.G + g];
      to = base + rank;
      if (rank == 0) at[wave * p.G + g] = base + __popcll(same);
      // (always, unless another call writes to the workspace meanwhile)
      if (is_place(to, p.R)) p.rows[to] = (int)i;
      else to = -1;
    }
    asm volatile("" ::: "memory");   // the wave's own writes, then its own reads: in order
    if (i < mine_end) {
      p.slots[i] = to;
      if (i >= total) p.rows[i] = -1;      // behind the last group
    }
  }
}

// ------------------------------------------------------------ the weighted sum

// 8 columns a thread; up to eight of the token's rows are loaded before any is added.
// Bound by HBM: 4632 tokens of 8 rows of 7168 and a shared one, 664 MB, 129 us, as
// fast as a copy; 16 tokens 4.4 us, most of it a launch.
__global__ __launch_bounds__(256)
void moe_combine_kernel(MoeCombineArgs p) {
  const int64_t m = blockIdx.x / p.parts;
  const int64_t c = ((int64_t)(blockIdx.x % p.parts) * 256 + threadIdx.x) * 8;
  if (c >= p.d) return;
  float acc[8] = {};
  layer::v4u own = {0u, 0u, 0u, 0u};
  if (p.shared) own = *reinterpret_cast<const layer::v4u*>(p.shared + m * p.lds + c);
  for (int j0 = 0; j0 < p.top; j0 += 8) {
    layer::v4u y[8];
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int slot = j0 + j < p.top ? p.slots[m * p.top + j0 + j] : -1;
      y[j] = layer::v4u{0u, 0u, 0u, 0u};
      w[j] = 0.f;
      if (slot >= 0 && slot < p.R) {
        w[j] = p.weights[m * p.top + j0 + j];
        y[j] = *reinterpret_cast<const layer::v4u*>(p.y + slot * p.ldy + c);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] += w[j] * layer::bf16_lo(y[j][i]);
        acc[2 * i + 1] += w[j] * layer::bf16_hi(y[j][i]);
      }
  }
  layer::v4u o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = layer::pack_bf16(acc[2 * i] + layer::bf16_lo(own[i]), acc[2 * i + 1] + layer::bf16_hi(own[i]));
  *reinterpret_cast<layer::v4u*>(p.out + m * p.ldo + c) = o;
}

}  // namespace

hipError_t launch_moe_route(const MoeRouteArgs& p, hipStream_t stream) {
  // A wave a token takes less time where tokens are few, a row of 16 lanes fewer
  // instructions (us, top 8, without a bias, wave / row: 64 experts, 4632 tokens 4.5 / 4.0,
  // 8192 5.8 / 4.1; 128 experts, 8192 6.6 / 5.5; 256 experts, 16384 14.3 / 12.0; with a bias
  // 6.9 / 4.8, 9.4 / 5.0, 7.9 / 7.3, 19.6 / 19.8).
  const bool rows = p.E <= 256 && p.top <= 16 && p.M >= 40 * (int64_t)p.E;
  const int64_t blocks = rows ? (p.M + 15) / 16 : (p.M + 3) / 4;
  const auto kern = rows ? (p.E <= 16    ? moe_route_kernel<16, 1>
                            : p.E <= 32  ? moe_route_kernel<16, 2>
                            : p.E <= 64  ? moe_route_kernel<16, 4>
                            : p.E <= 128 ? moe_route_kernel<16, 8>
                                         : moe_route_kernel<16, 16>)
                    : p.E <= 64  ? moe_route_kernel<64, 1>
                    : p.E <= 128 ? moe_route_kernel<64, 2>
                    : p.E <= 256 ? moe_route_kernel<64, 4>
                    : p.E <= 512 ? moe_route_kernel<64, 8>
                                 : moe_route_kernel<64, 16>;
  hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(256), 0, stream, p);
  return hipGetLastError();
}

// Entries of a workgroup, of which there are at most GROUP_CHUNKS. An entry a thread
// (two: 1024 entries 4.6 us for 3.8, 16384 7.8 for 6.9).
int64_t group_rows_chunk(int64_t R) {
  const int64_t share = (R + GROUP_CHUNKS - 1) / GROUP_CHUNKS;
  return share <= 1024 ? 1024 : (share + SORT_THREADS - 1) / SORT_THREADS * SORT_THREADS;
}

// Chunks that a launch of their own counts; 0 where every workgroup counts all
// entries itself (us, itself / a launch, 256 groups: 2048 entries 4.2 / 5.8, 8192 5.4 /
// 6.6, 12000 6.6 / 6.7, 16384 7.5 / 6.6).
int64_t group_rows_counts(int64_t R) {
  const int64_t chunk = group_rows_chunk(R), chunks = (R + chunk - 1) / chunk;
  return chunks > 8 ? chunks : 0;
}

hipError_t launch_group_rows(GroupRowsArgs p, hipStream_t stream) {
  p.chunk = group_rows_chunk(p.R);
  int64_t chunks = (p.R + p.chunk - 1) / p.chunk;
  if (chunks < 1) chunks = 1;
  if (group_rows_counts(p.R) == 0) p.counts = nullptr;
  if (p.counts) {
    hipLaunchKernelGGL(group_count_kernel, dim3((unsigned)chunks), dim3(SORT_THREADS), 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(group_place_kernel, dim3((unsigned)chunks), dim3(SORT_THREADS), 0, stream, p);
  return hipGetLastError();
}

int32_t moe_combine_parts(int64_t d) { return (int32_t)((d + 2047) / 2048); }

hipError_t launch_moe_combine(MoeCombineArgs p, hipStream_t stream) {
  p.parts = moe_combine_parts(p.d);
  hipLaunchKernelGGL(moe_combine_kernel, dim3((unsigned)(p.M * p.parts)), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace iqp
