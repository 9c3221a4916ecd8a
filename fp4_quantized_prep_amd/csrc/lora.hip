// Low-rank adapters beside a shared projection, for rows sorted by adapter:
//   out[m] += s_g B_g (A_g x[m]),  A_g [r, K], B_g [N, r], m's adapter g
// in two launches: h = A_g x (the first kernel, cut along K where there are few
// rows, each piece's sums kept apart in float32), then out += s_g B_g h.
#include "layer_common.h"
#include "row_groups.h"

namespace iqp {
namespace {

using layer::v4f;
using layer::v4u;
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int LORA_ROWS = 64;     // places of a workgroup
constexpr int LORA_COLS = 256;    // output columns of a workgroup (four waves of 64)

__device__ __forceinline__ v8bf operand(v4u v) { return __builtin_bit_cast(v8bf, v); }

__device__ __forceinline__ int64_t row_of(const LoraArgs& p, const groups::Tile& t, int r) {
  if (r >= t.rows) return -1;
  const int m = p.groups.rows[t.begin + r];
  return m >= 0 && m < p.M ? m : -1;
}

// h[z, place, i] = sum of A[g, i, k] x[m, k] over piece z of K. 16x16x32 MFMA: rows
// of A as its rows, places as its columns; operands straight from memory, 64 k a
// step. Up to 16 places: the four waves share out the steps and their sums meet in
// LDS; more: each wave takes 16 of them.
template <int RT>
__global__ __launch_bounds__(256)
void lora_shrink_kernel(LoraArgs p) {
  constexpr int PITCH = 16 * RT + 4;
  __shared__ __attribute__((aligned(16))) float part[4 * 16 * PITCH];
  const groups::Tile t = groups::find_tile(p.groups, LORA_ROWS, p.splits, groups::item_of(blockIdx.x, 1));
  if (t.rows <= 0) return;
  const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool few = t.rows <= 16;
  const int r0 = few ? 0 : 16 * wave;
  if (r0 >= t.rows) return;            // (more than 16 rows: no barrier below)
  const int64_t m = row_of(p, t, r0 + col);
  const uint16_t* const x = p.x + (m < 0 ? 0 : m) * p.ldx;      // columns of rows that are none are not kept
  const uint16_t* a[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int r = 16 * i + col < p.rank ? 16 * i + col : p.rank - 1;      // likewise
    a[i] = p.a + ((int64_t)t.group * p.rank + r) * p.K;
  }
  const int steps = (int)((p.K + 63) / 64);
  const int first = (int)((int64_t)steps * t.part / p.splits), last = (int)((int64_t)steps * (t.part + 1) / p.splits);
  v4f acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
  const v4u zero = {0u, 0u, 0u, 0u};
#pragma unroll 2
  for (int s = few ? first + wave : first; s < last; s += few ? 4 : 1) {
    v4u fx[2], fa[2][RT];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t k = 64 * (int64_t)s + 32 * h + 8 * g;
      const bool in = k < p.K;
      fx[h] = in ? *reinterpret_cast<const v4u*>(x + k) : zero;
#pragma unroll
      for (int i = 0; i < RT; ++i) fa[h][i] = in ? *reinterpret_cast<const v4u*>(a[i] + k) : zero;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < RT; ++i) acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand(fa[h][i]), operand(fx[h]), acc[i], 0, 0, 0);
  }
  float* const to = p.h + ((int64_t)t.part * p.groups.R + t.begin) * (16 * RT);
  if (!few) {
    if (r0 + col < t.rows)
#pragma unroll
      for (int i = 0; i < RT; ++i) *reinterpret_cast<v4f*>(to + (r0 + col) * (16 * RT) + 16 * i + 4 * g) = acc[i];
    return;
  }
#pragma unroll
  for (int i = 0; i < RT; ++i) *reinterpret_cast<v4f*>(part + (16 * wave + col) * PITCH + 16 * i + 4 * g) = acc[i];
  __syncthreads();
  for (int i = threadIdx.x; i < t.rows * 4 * RT; i += 256) {
    const int r = i / (4 * RT), c = 4 * (i % (4 * RT));
    v4f sum = *reinterpret_cast<const v4f*>(part + r * PITCH + c);
#pragma unroll
    for (int w = 1; w < 4; ++w) {
      const v4f v = *reinterpret_cast<const v4f*>(part + (16 * w + r) * PITCH + c);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += v[e];
    }
    *reinterpret_cast<v4f*>(to + r * (16 * RT) + c) = sum;
  }
}

// out += s B h. MFMA: rows of B as its rows, places as its columns; row 4 g + i of
// tile t is column 16 g + 4 t + i of the wave's 64, so that a lane has sixteen
// consecutive ones of one place. h goes in as two bf16 parts (16 significant
// bits together): the second product costs less than the output's way to memory,
// and h rounded to one would be off as much as the output's own rounding.
template <int KT>
__global__ __launch_bounds__(256)
void lora_expand_kernel(LoraArgs p) {
  const groups::Tile t = groups::find_tile(p.groups, LORA_ROWS, p.parts, groups::item_of(blockIdx.x, 1));
  if (t.rows <= 0) return;
  const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)t.part * LORA_COLS + 64 * wave;
  if (n0 >= p.N) return;
  const v4u zero = {0u, 0u, 0u, 0u};
  v4u b[KT][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int64_t n = n0 + 16 * (col >> 2) + 4 * i + (col & 3);
    n = n < p.N ? n : p.N - 1;         // columns past the last one are not kept
    const uint16_t* const row = p.b + (t.group * p.N + n) * p.rank;
#pragma unroll
    for (int s = 0; s < KT; ++s) b[s][i] = 32 * s + 8 * g < p.rank ? *reinterpret_cast<const v4u*>(row + 32 * s + 8 * g) : zero;
  }
  const float scale = p.scales ? p.scales[t.group] : 1.f;
  const int64_t n = n0 + 16 * g;
  for (int r0 = 0; r0 < t.rows; r0 += 16) {
    const int64_t m = row_of(p, t, r0 + col);
    const float* const h = p.h + ((int64_t)t.begin + (r0 + col < t.rows ? r0 + col : 0)) * p.h_pitch;
    v4f acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < KT; ++s) {
      const int k = 32 * s + 8 * g;
      v8bf hi, lo;
#pragma unroll
      for (int e = 0; e < 8; ++e) hi[e] = lo[e] = (__bf16)0.f;
      if (k < p.rank) {
        float v[8] = {};
        for (int z = 0; z < p.splits; ++z) {
          const float* const q = h + (int64_t)z * p.groups.R * p.h_pitch + k;
          const v4f v0 = *reinterpret_cast<const v4f*>(q), v1 = *reinterpret_cast<const v4f*>(q + 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] += v0[e];
            v[4 + e] += v1[e];
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = v[e] * scale;
          hi[e] = (__bf16)x;
          lo[e] = (__bf16)(x - (float)hi[e]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand(b[s][i]), lo, acc[i], 0, 0, 0);
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand(b[s][i]), hi, acc[i], 0, 0, 0);
      }
    }
    if (m < 0) continue;
    uint16_t* const out = p.out + m * p.ldo + n;
    if (p.wide_out && n + 16 <= p.N) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const v4u o = *reinterpret_cast<const v4u*>(out + 8 * c);
        v4u d;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          d[e] = layer::pack_bf16(layer::bf16_lo(o[e]) + acc[2 * c + e / 2][2 * (e & 1)],
                                  layer::bf16_hi(o[e]) + acc[2 * c + e / 2][2 * (e & 1) + 1]);
        *reinterpret_cast<v4u*>(out + 8 * c) = d;
      }
    } else {
#pragma unroll
      for (int c = 0; c < 16; ++c)
        if (n + c < p.N) out[c] = (uint16_t)layer::pack_bf16(layer::bf16_lo(out[c]) + acc[c / 4][c & 3], 0.f);
    }
  }
}

int64_t tiles_of(const RowGroups& g) { return g.R / LORA_ROWS + (g.G < g.R ? g.G : g.R); }

}  // namespace

// Pieces of K: enough that the first launch has 512 workgroups, of eight steps at least
int lora_splits(int64_t R, int32_t G, int64_t K) {
  const int64_t tiles = tiles_of(RowGroups{nullptr, nullptr, R, G}), steps = (K + 63) / 64;
  int64_t z = 512 / (tiles > 0 ? tiles : 1);
  if (z > steps / 8) z = steps / 8;
  return z < 1 ? 1 : z > 8 ? 8 : (int)z;
}

int lora_pitch(int32_t rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

hipError_t launch_lora_add(LoraArgs p, hipStream_t stream) {
  p.h_pitch = lora_pitch(p.rank);
  p.parts = (int32_t)((p.N + LORA_COLS - 1) / LORA_COLS);
  const int64_t tiles = tiles_of(p.groups);
  const int64_t shrink = (tiles * p.splits + 7) / 8 * 8, expand = (tiles * p.parts + 7) / 8 * 8;
  if (shrink > 0x7FFFFFFF || expand > 0x7FFFFFFF) return hipErrorInvalidValue;
  const auto first = p.h_pitch == 16 ? lora_shrink_kernel<1> : p.h_pitch == 32 ? lora_shrink_kernel<2> : p.h_pitch == 64 ? lora_shrink_kernel<4> : lora_shrink_kernel<8>;
  hipLaunchKernelGGL(first, dim3((unsigned)shrink), dim3(256), 0, stream, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const auto second = p.rank <= 32 ? lora_expand_kernel<1> : p.rank <= 64 ? lora_expand_kernel<2> : lora_expand_kernel<4>;
  hipLaunchKernelGGL(second, dim3((unsigned)expand), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace iqp
