// Around the products by expert: the router's choice of experts, the entries of
// a batch sorted by group, and every token's weighted sum of its experts' rows.
#include "iqprep.h"
#include "layer_common.h"
#include "row_groups.h"

namespace iqp {
namespace {

// ---------------------------------------------------------------- the router

// A float64 as an unsigned integer of the same order, NaN above all (zeros of
// either sign alike); never 0.
__device__ __forceinline__ uint64_t order_of(double v) {
  if (v != v) return ~0ull;
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return b >> 63 ? ~b : b | 1ull << 63;
}

template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t dpp_max(uint64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xF, false);
  const uint64_t o = (uint64_t)hi << 32 | lo;
  return o > v ? o : v;
}

// the largest of the 64 lanes, in every lane
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
  v = dpp_max<0x111, 0xF>(v);
  v = dpp_max<0x112, 0xF>(v);
  v = dpp_max<0x114, 0xF>(v);
  v = dpp_max<0x118, 0xF>(v);
  v = dpp_max<0x142, 0xA>(v);
  v = dpp_max<0x143, 0xC>(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, 63);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), 63);
  return (uint64_t)hi << 32 | lo;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

__device__ __forceinline__ double score_of(double z, int scoring) {
  if (scoring == IQP_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-z));
  return sqrt((z > 0.0 ? z : 0.0) + log1p(exp(-fabs(z))));    // sqrt of softplus
}

// A wave a token, expert 64 v + lane its lane's v-th value. Scores and choices are
// float64, so that which expert is taken does not hang on how an exponential is
// rounded; the order is by choice, then by index.
template <int VPL>
__global__ __launch_bounds__(256)
void moe_route_kernel(MoeRouteArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t m = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (m >= p.M) return;
  const auto logit = [&](int e) __attribute__((always_inline)) {
    return p.half ? (double)__uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p.logits)[m * p.ld + e] << 16)
                  : (double)reinterpret_cast<const float*>(p.logits)[m * p.ld + e];
  };
  const double NONE = -__builtin_inf();
  double z[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) z[v] = 64 * v + lane < p.E ? logit(64 * v + lane) : NONE;
  double top = 0.0, sum = 1.0;     // of softmax over all experts, where that is asked for
  if (p.scoring == IQP_SCORE_SOFTMAX && (p.bias || !p.renormalize)) {
    top = NONE;
#pragma unroll
    for (int v = 0; v < VPL; ++v) top = z[v] > top ? z[v] : top;
#pragma unroll
    for (int d = 32; d; d >>= 1) {
      const double o = __shfl_xor(top, d);
      top = o > top ? o : top;
    }
    sum = 0.0;
#pragma unroll
    for (int v = 0; v < VPL; ++v) sum += z[v] == NONE ? 0.0 : exp(z[v] - top);
    sum = wave_sum(sum);
  }
  uint64_t key[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int e = 64 * v + lane;
    double c = z[v];
    if (p.bias && e < p.E && c != NONE)
      c = (p.scoring == IQP_SCORE_SOFTMAX ? exp(c - top) / sum : score_of(c, p.scoring)) + (double)p.bias[e];
    key[v] = e < p.E ? order_of(c) : 0;
  }
  int mine = 0;      // lane j: the j-th expert
  for (int j = 0; j < p.top; ++j) {
    uint64_t best = key[0];
    int at = 0;
#pragma unroll
    for (int v = 1; v < VPL; ++v)
      if (key[v] > best) {
        best = key[v];
        at = v;
      }
    const uint64_t most = wave_max(best);
    uint64_t who = __ballot(best == most);
    int e = 64 * at + lane, lead = __ffsll((unsigned long long)who) - 1;
    // lanes with the same choice: the lowest index has the lowest v, then the lowest lane
    for (uint64_t rest = who & (who - 1); rest; rest &= rest - 1) {
      const int other = __ffsll((unsigned long long)rest) - 1;
      if (__builtin_amdgcn_readlane(at, other) < __builtin_amdgcn_readlane(at, lead)) lead = other;
    }
    e = __builtin_amdgcn_readlane(e, lead);
    if (lane == lead)
#pragma unroll
      for (int v = 0; v < VPL; ++v) key[v] = v == at ? 0 : key[v];
    mine = lane == j ? e : mine;
  }
  double w = 0.0;
  const double zs = logit(mine);
  if (p.scoring == IQP_SCORE_SOFTMAX) {
    if (!p.bias && p.renormalize) {
      const double first = __shfl(zs, 0);      // the largest logit
      w = zs == NONE ? 0.0 : exp(zs - first);
    } else {
      w = zs == NONE ? 0.0 : exp(zs - top) / sum;
    }
  } else {
    w = score_of(zs, p.scoring);
  }
  w = lane < p.top ? w : 0.0;
  if (p.renormalize) {
    const double total = wave_sum(w);
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
// of its group before it in its wave.
__global__ __launch_bounds__(SORT_THREADS)
void group_place_kernel(GroupRowsArgs p) {
  __shared__ int at[SORT_WAVES * MAX_GROUPS];
  __shared__ int sums[SORT_WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t first = (int64_t)blockIdx.x * p.chunk, end = first + p.chunk < p.R ? first + p.chunk : p.R;
  const int64_t share = ((p.chunk + SORT_THREADS - 1) / SORT_THREADS) * 64;      // entries of a wave
  const int64_t mine = first + wave * share, mine_end = mine + share < end ? mine + share : end;
  for (int g = tid; g < SORT_WAVES * p.G; g += SORT_THREADS) at[g] = 0;
  __syncthreads();
  for (int64_t i = mine + lane; i < mine_end; i += 64) {
    const int g = group_of(p, i);
    if (g < p.G) atomicAdd(&at[wave * p.G + g], 1);
  }
  __syncthreads();
  // thread g: its group's entries before this chunk, and in all
  int before = 0, all = 0;
  if (tid < p.G) {
    if (gridDim.x == 1) {
#pragma unroll
      for (int w = 0; w < SORT_WAVES; ++w) all += at[w * p.G + tid];
    } else {
      for (unsigned c = 0; c < gridDim.x; ++c) {
        const int n = p.counts[(int64_t)c * p.G + tid];
        before += c < blockIdx.x ? n : 0;
        all += n;
      }
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
    const int g = i < mine_end ? group_of(p, i) : p.G;
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
      p.rows[to] = (int)i;
    }
    if (i < mine_end) {
      p.slots[i] = to;
      if (i >= total) p.rows[i] = -1;      // behind the last group
    }
  }
}

// ------------------------------------------------------------ the weighted sum

// 8 columns a thread; up to eight of the token's rows are loaded before any is added
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
  const int64_t blocks = (p.M + 3) / 4;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  const auto kern = p.E <= 64    ? moe_route_kernel<1>
                    : p.E <= 128 ? moe_route_kernel<2>
                    : p.E <= 256 ? moe_route_kernel<4>
                    : p.E <= 512 ? moe_route_kernel<8>
                                 : moe_route_kernel<16>;
  hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(256), 0, stream, p);
  return hipGetLastError();
}

// entries of a workgroup: at most GROUP_CHUNKS of them
int64_t group_rows_chunk(int64_t R) {
  const int64_t share = (R + GROUP_CHUNKS - 1) / GROUP_CHUNKS;
  return share <= 2048 ? 2048 : (share + SORT_THREADS - 1) / SORT_THREADS * SORT_THREADS;
}

hipError_t launch_group_rows(GroupRowsArgs p, hipStream_t stream) {
  p.chunk = group_rows_chunk(p.R);
  int64_t chunks = (p.R + p.chunk - 1) / p.chunk;
  if (chunks < 1) chunks = 1;
  if (chunks > 1) {
    hipLaunchKernelGGL(group_count_kernel, dim3((unsigned)chunks), dim3(SORT_THREADS), 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(group_place_kernel, dim3((unsigned)chunks), dim3(SORT_THREADS), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_moe_combine(MoeCombineArgs p, hipStream_t stream) {
  p.parts = (int32_t)((p.d + 2047) / 2048);
  const int64_t blocks = p.M * p.parts;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL(moe_combine_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace iqp
