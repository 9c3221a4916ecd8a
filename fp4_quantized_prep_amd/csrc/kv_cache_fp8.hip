// The FP8 key/value cache: bf16 keys and values quantised to E4M3 as they are
// written, and read back as bf16.
//
// Layout. A block holds B tokens (a power of two, 16 to 128) of one layer:
//   keys    E4M3 [n_blocks, Hk, B, D], a token's D values together;
//   values  E4M3 [n_blocks, Hk, D, B], a dim's B tokens together, which is the
//           order in which attention's second product reads them;
//   scales  one UE8M0 byte per block and head for the keys, one for the values:
//           value = code * 2^(byte - 127).
//
// Writing. The exponent of a block is the one the 1x128 quantizer would choose
// for all the values written into it at once, e = max(ceil(log2(amax / 448)),
// -22): a write that covers the block's first token starts afresh, a later one
// keeps the larger of the block's exponent and its own. Where that raises it,
// the codes of the block's earlier tokens are divided by the power of two and
// rounded to E4M3 again, which is exact unless a code falls among the
// subnormals. Nobody else writes those bytes: one workgroup has a block and
// head of one sequence to itself, for its keys and its values.
//
// HBM-bound (2 bytes in and 1 out a value). The workgroup holds its new rows in
// registers (16 bytes a lane) from the amax to the conversion, so they are read
// once; the values are turned in LDS, and a piece of 16 tokens that is partly new
// is merged with its old codes and stored whole.
//
// Measured: three prompts of 900 to 4632 tokens after up to 700, 8 heads of 128: 22.4 us
// for writing and reading back, 4.5 TB/s (a large copy reaches 5.1); a token each
// for 64 sequences: 7.0 us, four dependent loads (lengths, block table, rows and
// scales, old codes) and a launch.
#include "fp8_block.h"
#include "layer_common.h"

namespace iqp {
namespace {

using namespace layer;

constexpr int KV_THREADS = 256;
constexpr int MAX_B = 128;
constexpr int PAD = 4;              // bytes between the turned rows in LDS

// A workgroup's share: rows [lo, hi) of block `block`, the first of them row
// `row` of the batch.
struct Share {
  int64_t block;
  int64_t row;
  int lo, hi;
};

// Item -> sequence and block (see find_sequence: a sequence of n rows touches
// at most floor((n - 2) / B) + 2 blocks). False where the item has no rows. The
// block is as the table has it: held(..) says whether the cache has it, asked
// only after the loads that do not need it are on their way.
__device__ __forceinline__ bool find_share(const SeqBatch& b, int64_t item, Share& out) {
  const SeqRows q = find_sequence(b, item, 1, b.log_block, 2);
  const int n = q.end - q.begin;
  if (n <= 0 || q.len <= 0) return false;
  const int64_t first = (int64_t)q.len - n;       // position of the first row (rows before position 0: left out)
  const int64_t idx = (first >> b.log_block) + item - item_key(q, 1, b.log_block, 2);
  const int64_t base = idx << b.log_block;
  if (idx < 0 || idx >= b.max_blocks || base >= q.len) return false;
  out.lo = first > base ? (int)(first - base) : 0;
  out.hi = q.len - base < ((int64_t)1 << b.log_block) ? (int)(q.len - base) : 1 << b.log_block;
  if (out.lo >= out.hi) return false;
  out.row = q.begin + (base + out.lo - first);
  out.block = b.table[(int64_t)q.s * b.ld_table + idx];
  return true;
}

__device__ __forceinline__ bool held(const SeqBatch& b, int64_t block) { return block >= 0 && block < b.n_blocks; }

// four E4M3 codes times mul (a power of two <= 1), rounded to E4M3
__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float mul) {
  const v2f a = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, true);
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a[0] * mul, a[1] * mul, 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(b[0] * mul, b[1] * mul, r, true);
  return (uint32_t)r;
}

// the bytes of a dword below n
__device__ __forceinline__ uint32_t byte_mask(int n) { return n >= 4 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << (8 * n)) - 1u; }

// eight E4M3 codes times mul, as bf16
__device__ __forceinline__ v4u widen8(v2u c, float mul) {
  v4u o;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const v2f a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[j], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[j], true);
    o[2 * j] = pack_bf16(a[0] * mul, a[1] * mul);
    o[2 * j + 1] = pack_bf16(b[0] * mul, b[1] * mul);
  }
  return o;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = fp8q::lanes16_max(v);
  v = max(v, (uint32_t)__shfl_xor((int)v, 16));
  return max(v, (uint32_t)__shfl_xor((int)v, 32));
}

template <int D>
__global__ __launch_bounds__(KV_THREADS)
void kv_append_kernel(KvAppendArgs p) {
  constexpr int LANES = D / 8;                    // lanes of a row
  constexpr int ROWS = KV_THREADS / LANES;        // rows of a pass
  constexpr int PASSES = MAX_B / ROWS;
  __shared__ __attribute__((aligned(16))) uint8_t turned[D * (MAX_B + PAD)];
  __shared__ uint32_t part[2][KV_THREADS / 64];

  Share sh;
  if (!find_share(p.seq, blockIdx.x, sh)) return;   // uniform over the workgroup
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int head = blockIdx.y;
  const int B = 1 << p.seq.log_block;
  const int l = tid % LANES, r0 = tid / LANES;
  const int n = sh.hi - sh.lo;

  v4u x[2][PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int r = r0 + ROWS * i;
    x[0][i] = x[1][i] = v4u{0u, 0u, 0u, 0u};
    if (r < n) {
      x[0][i] = *reinterpret_cast<const v4u*>(p.k + (sh.row + r) * p.ldk + (int64_t)head * D + 8 * l);
      x[1][i] = *reinterpret_cast<const v4u*>(p.v + (sh.row + r) * p.ldv + (int64_t)head * D + 8 * l);
    }
  }
  if (!held(p.seq, sh.block)) return;               // uniform over the workgroup
  const int64_t slot = sh.block * p.Hk + head;
  uint8_t* const kb = p.k_cache + slot * B * D;
  uint8_t* const vb = p.v_cache + slot * B * D;
  int old[2] = {0, 0};
  if (sh.lo > 0) {
    old[0] = (int)p.k_scales[slot] - 127;
    old[1] = (int)p.v_scales[slot] - 127;
  }
  // 16 tokens of a value dim, c of them from c0 to c1, are a piece; the thread's
  // first one, if it holds codes that stay: on its way while the maximum is found
  const int c0 = sh.lo >> 4, c1 = (sh.hi + 15) >> 4;
  v4u kept = {0u, 0u, 0u, 0u};
  {
    const int c = c0 + tid % (c1 - c0), d = tid / (c1 - c0);
    if (d < D && (sh.lo > 16 * c || sh.hi < 16 * c + 16)) kept = *reinterpret_cast<const v4u*>(vb + d * B + 16 * c);
  }
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
      a = max(a, max(max(fp8q::mag2(x[m][i][0]), fp8q::mag2(x[m][i][1])),
                     max(fp8q::mag2(x[m][i][2]), fp8q::mag2(x[m][i][3]))));
    a = wave_max(a);
    if (lane == 0) part[m][wave] = a;
  }
  __syncthreads();
  int e[2];
  bool grown[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    uint32_t a = part[m][0];
#pragma unroll
    for (int w = 1; w < KV_THREADS / 64; ++w) a = max(a, part[m][w]);
    e[m] = fp8q::block_exponent(a);
    grown[m] = sh.lo > 0 && e[m] > old[m];
    if (sh.lo > 0) e[m] = max(e[m], old[m]);
    e[m] = min(e[m], 126);                          // 2^-e stays a normal float whatever byte was there
  }
  if (tid == 0) {
    p.k_scales[slot] = (uint8_t)(e[0] + 127);
    p.v_scales[slot] = (uint8_t)(e[1] + 127);
  }

  // keys: the new rows, then the earlier ones where the exponent grew
  const float km = pow2(-e[0]), vm = pow2(-e[1]);
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int r = r0 + ROWS * i;
    if (r < n) {
      *reinterpret_cast<v2u*>(kb + (sh.lo + r) * D + 8 * l) =
          v2u{fp8q::cvt4(x[0][i][0], x[0][i][1], km), fp8q::cvt4(x[0][i][2], x[0][i][3], km)};
      const v2u c = {fp8q::cvt4(x[1][i][0], x[1][i][1], vm), fp8q::cvt4(x[1][i][2], x[1][i][3], vm)};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        turned[(8 * l + j) * (MAX_B + PAD) + sh.lo + r] = (uint8_t)(c[j >> 2] >> (8 * (j & 3)));
    }
  }
  if (grown[0]) {
    const float mul = pow2(max(old[0] - e[0], -126));
    for (int i = tid; i < sh.lo * (D / 16); i += KV_THREADS) {
      v4u c = *reinterpret_cast<const v4u*>(kb + 16 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] = rescale4(c[j], mul);
      *reinterpret_cast<v4u*>(kb + 16 * i) = c;
    }
  }
  __syncthreads();
  // values, piece by piece: what is neither new nor rescaled goes back as it was
  const float mul = grown[1] ? pow2(max(old[1] - e[1], -126)) : 1.f;
  const int first = grown[1] ? 0 : c0;              // the first piece that is written
  for (int i = tid; i < D * (c1 - first); i += KV_THREADS) {
    const int c = first + i % (c1 - first), d = i / (c1 - first);
    uint8_t* const dst = vb + d * B + 16 * c;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(turned + d * (MAX_B + PAD) + 16 * c);
    const int a = sh.lo - 16 * c, z = sh.hi - 16 * c;     // bytes [a, z) are new
    v4u w = {src[0], src[1], src[2], src[3]};
    if (a > 0 || z < 16) {
      const v4u o = i == tid && !grown[1] ? kept : *reinterpret_cast<const v4u*>(dst);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t below = byte_mask(a - 4 * j), upto = byte_mask(z - 4 * j);
        const uint32_t g = grown[1] ? rescale4(o[j], mul) : o[j];
        w[j] = (g & below) | (w[j] & upto & ~below) | (o[j] & ~upto);
      }
    }
    *reinterpret_cast<v4u*>(dst) = w;
  }
}

template <int D>
__global__ __launch_bounds__(KV_THREADS)
void kv_read_kernel(KvReadArgs p) {
  constexpr int LANES = D / 8;
  constexpr int ROWS = KV_THREADS / LANES;
  __shared__ __attribute__((aligned(16))) uint8_t turned[D * (MAX_B + PAD)];
  const int tid = threadIdx.x;
  const int head = blockIdx.y;
  Share sh;
  if (!find_share(p.seq, blockIdx.x, sh) || !held(p.seq, sh.block)) return;   // uniform over the workgroup
  const int B = 1 << p.seq.log_block;
  const int64_t slot = sh.block * p.Hk + head;
  const uint8_t* const kb = p.k_cache + slot * B * D;
  const uint8_t* const vb = p.v_cache + slot * B * D;
  const int ke = min(max((int)p.k_scales[slot] - 127, -126), 127), ve = min(max((int)p.v_scales[slot] - 127, -126), 127);
  const float km = pow2(ke), vm = pow2(ve);
  const int c0 = sh.lo >> 4, c1 = (sh.hi + 15) >> 4;
  for (int i = tid; i < D * (c1 - c0); i += KV_THREADS) {
    const int c = c0 + i % (c1 - c0), d = i / (c1 - c0);
    const v4u w = *reinterpret_cast<const v4u*>(vb + d * B + 16 * c);
    uint32_t* dst = reinterpret_cast<uint32_t*>(turned + d * (MAX_B + PAD) + 16 * c);
#pragma unroll
    for (int j = 0; j < 4; ++j) dst[j] = w[j];
  }
  __syncthreads();
  const int l = tid % LANES;
  for (int r = sh.lo + tid / LANES; r < sh.hi; r += ROWS) {
    const int64_t row = sh.row + (r - sh.lo);
    const v2u kc = *reinterpret_cast<const v2u*>(kb + r * D + 8 * l);
    v2u vc = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      vc[j >> 2] |= (uint32_t)turned[(8 * l + j) * (MAX_B + PAD) + r] << (8 * (j & 3));
    *reinterpret_cast<v4u*>(p.k_out + row * p.ldk + (int64_t)head * D + 8 * l) = widen8(kc, km);
    *reinterpret_cast<v4u*>(p.v_out + row * p.ldv + (int64_t)head * D + 8 * l) = widen8(vc, vm);
  }
}

// work items: floor(T / B) + 2 S bound the blocks that the sequences touch
int64_t items_of(const SeqBatch& b) { return (b.T >> b.log_block) + 2 * (int64_t)b.S; }

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs& p, int D, hipStream_t stream) {
  const int64_t items = items_of(p.seq);
  if (items > 0x7FFFFFFF) return hipErrorInvalidValue;
  auto kern = D == 64 ? kv_append_kernel<64> : kv_append_kernel<128>;
  hipLaunchKernelGGL(kern, dim3((unsigned)items, (unsigned)p.Hk), dim3(KV_THREADS), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvReadArgs& p, int D, hipStream_t stream) {
  const int64_t items = items_of(p.seq);
  if (items > 0x7FFFFFFF) return hipErrorInvalidValue;
  auto kern = D == 64 ? kv_read_kernel<64> : kv_read_kernel<128>;
  hipLaunchKernelGGL(kern, dim3((unsigned)items, (unsigned)p.Hk), dim3(KV_THREADS), 0, stream, p);
  return hipGetLastError();
}

}  // namespace iqp
