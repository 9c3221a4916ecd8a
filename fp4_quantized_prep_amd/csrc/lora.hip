// Low-rank adapters beside a shared projection, for rows sorted by adapter:
//   out[m] += s_g B_g (A_g x[m]),  A_g [r, K], B_g [N, r], m's adapter g
// in two launches: h = A_g x (the first kernel, cut along K where there are few
// rows, each piece's sums kept apart in float32), then out += s_g B_g h.
//
// The second is bound by out's way from and to memory (4632x8192, rank 64: 33 us for
// 30 at a copy's rate), the first by A's way from L2, once for every 16 or 32 rows (K
// 1536: 8 us); few rows by two launches and what they wait for one after the other (64
// tokens of 32 adapters, 1536x7168, rank 16: 4.2 and 4.2 us for 10 MB).
#include "iq_common.h"
#include "layer_common.h"
#include "row_groups.h"

namespace iqp {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int SHRINK_WAVES = 4;   // first launch: waves of a workgroup
constexpr int LORA_ROWS = 64;     // second launch: places of a workgroup
constexpr int LORA_COLS = 256;    // output columns of a workgroup (four waves of 64)

// An offset beyond every buffer: they reach less than 2^31 bytes. Joined to others
// by "or", so that two of them stay one.
constexpr uint32_t PAST = 0x80000000u;

constexpr int waitcnt_vm(int n) { return (n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14); }

__device__ __forceinline__ v8bf operand(v4u v) { return __builtin_bit_cast(v8bf, v); }

// the row of place r of the tile, -1 where there is none
__device__ __forceinline__ int64_t row_of(const LoraArgs& p, const groups::Tile& t, int r) {
  const int m = p.groups.rows[t.begin + (r < t.rows ? r : 0)];
  return r < t.rows && m >= 0 && m < p.M ? m : -1;
}

// h[z, place, i] = sum of A[g, i, k] x[m, k] over piece z of K, 16 MT places a
// workgroup. Its waves share out K in steps of 64 and stream them through LDS rings
// of their own (rows of 128 bytes, 16-byte chunk c of row r at c ^ r % 8, so that
// the operand reads meet distinct banks); their sums meet in LDS. 16x16x32 MFMA: rows
// of A as its rows, places as its columns. Operands straight from memory would take
// the address unit 64 cycles a load, a line for every lane, for the 16 of whole
// lines (4632x64x1536: 17.5 us, so 9.4).
template <int MT, int RT>
constexpr int shrink_stage() { return 2048 * (MT + RT); }

template <int MT, int RT, int NST>
__device__ __forceinline__ void shrink(const LoraArgs& p, uint8_t* lds) {
  constexpr int PITCH = 16 * RT + 4, STAGE = shrink_stage<MT, RT>(), NCOPY = 2 * (MT + RT);
  static_assert(4 * 16 * MT * PITCH <= NST * STAGE, "a wave's sums, in its ring's place");
  const groups::Tile t = groups::find_tile(p.groups, 16 * MT, p.splits, 1, groups::item_of(blockIdx.x, 1), false);
  if (t.rows <= 0) return;
  const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int steps = (int)((p.K + 63) / 64), K = (int)p.K;
  const int first = (int)((int64_t)steps * t.part / p.splits) + wave;
  const int last = (int)((int64_t)steps * (t.part + 1) / p.splits);
  const rsrc_t rx = make_rsrc(p.x, 2 * (uint64_t)((p.M - 1) * p.ldx + p.K));
  const rsrc_t ra = make_rsrc(p.a + (int64_t)t.group * p.rank * p.K, 2 * (uint64_t)p.rank * p.K);
  // copy c moves rows 8 c + lane / 8; rows that are none read zeros
  const int chunk = (lane & 7) ^ (lane >> 3 & 7);
  uint32_t vx[2 * MT], va[2 * RT];
#pragma unroll
  for (int c = 0; c < 2 * MT; ++c) {
    const int64_t m = row_of(p, t, 8 * c + (lane >> 3));
    vx[c] = m < 0 ? PAST : (uint32_t)(2 * (m * p.ldx + 8 * chunk));
  }
#pragma unroll
  for (int c = 0; c < 2 * RT; ++c) {
    const int r = 8 * c + (lane >> 3);
    va[c] = r < p.rank ? 2 * (uint32_t)(r * K + 8 * chunk) : PAST;
  }
  uint8_t* const ring = lds + wave * NST * STAGE;
  auto copy = [&](int s, int st) __attribute__((always_inline)) {
    // past the last column x reads zeros, and whatever A holds there goes with them
    const uint32_t past = s < last ? 0 : PAST, tail = 64 * s + 8 * chunk < K ? past : PAST;
    uint8_t* const b = ring + st * STAGE;
#pragma unroll
    for (int c = 0; c < 2 * MT; ++c)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void*)(b + 1024 * c), 16, (vx[c] + 128 * s) | tail, 0, 0, 0);
#pragma unroll
    for (int c = 0; c < 2 * RT; ++c)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(b + 1024 * (2 * MT + c)), 16, (va[c] + 128 * s) | past, 0, 0, 0);
  };
#pragma unroll
  for (int st = 0; st < NST; ++st) copy(first + st * SHRINK_WAVES, st);
  __builtin_amdgcn_sched_barrier(0);
  v4f acc[MT][RT];
#pragma unroll
  for (int u = 0; u < MT; ++u)
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[u][i] = v4f{0.f, 0.f, 0.f, 0.f};
  constexpr int WAIT = waitcnt_vm((NST - 1) * NCOPY);
  const int c0 = 128 * col + 16 * (g ^ (col & 7)), c1 = 128 * col + 16 * ((4 + g) ^ (col & 7));
  int st = 0;
  for (int s = first; s < last; s += SHRINK_WAVES) {
    __builtin_amdgcn_s_waitcnt(WAIT);
    asm volatile("" ::: "memory");
    const uint8_t* const b = ring + st * STAGE;
    v4u fx[MT][2], fa[RT][2];
#pragma unroll
    for (int u = 0; u < MT; ++u) {
      fx[u][0] = *reinterpret_cast<const v4u*>(b + 2048 * u + c0);
      fx[u][1] = *reinterpret_cast<const v4u*>(b + 2048 * u + c1);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      fa[i][0] = *reinterpret_cast<const v4u*>(b + 2048 * (MT + i) + c0);
      fa[i][1] = *reinterpret_cast<const v4u*>(b + 2048 * (MT + i) + c1);
    }
    // the stage is read: refill it
    __builtin_amdgcn_s_waitcnt(WAITCNT_LGKM0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    copy(s + NST * SHRINK_WAVES, st);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int u = 0; u < MT; ++u)
          acc[u][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand(fa[i][h]), operand(fx[u][h]), acc[u][i], 0, 0, 0);
    st = st + 1 < NST ? st + 1 : 0;
  }
  __builtin_amdgcn_s_waitcnt(WAITCNT_VM0);
  __syncthreads();
  float* const part = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int u = 0; u < MT; ++u)
#pragma unroll
    for (int i = 0; i < RT; ++i) *reinterpret_cast<v4f*>(part + (16 * (MT * wave + u) + col) * PITCH + 16 * i + 4 * g) = acc[u][i];
  __syncthreads();
  float* const to = p.h + ((int64_t)t.part * p.groups.R + t.begin) * (16 * RT);
  for (int i = threadIdx.x; i < t.rows * 4 * RT; i += 64 * SHRINK_WAVES) {
    const int r = i / (4 * RT), c = 4 * (i % (4 * RT));
    v4f sum = *reinterpret_cast<const v4f*>(part + r * PITCH + c);
#pragma unroll
    for (int w = 1; w < SHRINK_WAVES; ++w) {
      const v4f v = *reinterpret_cast<const v4f*>(part + (16 * MT * w + r) * PITCH + c);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += v[e];
    }
    *reinterpret_cast<v4f*>(to + r * (16 * RT) + c) = sum;
  }
}

template <int MT, int RT, int NST>
__global__ __launch_bounds__(64 * SHRINK_WAVES)
void lora_shrink_kernel(LoraArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[SHRINK_WAVES * NST * shrink_stage<MT, RT>()];
  shrink<MT, RT, NST>(p, lds);
}

// h of the tile's places, added up once for the workgroup and scaled, in two bf16
// parts (16 significant bits together: the second product costs less than the
// output's way to memory, and h rounded to one would be off as much as the output's
// own rounding). An infinite one is its high part alone. Eight values a thread and
// turn; `parts` rows of 64 KT + 8, the high parts first.
template <int KT>
__device__ __forceinline__ void split_h(const LoraArgs& p, const groups::Tile& t, __bf16* parts) {
  constexpr int HP = 64 * KT + 8;
  const float scale = p.scales ? p.scales[t.group] : 1.f;
  for (int c = threadIdx.x; c < t.rows * (4 * KT); c += 256) {
    const int r = c / (4 * KT), k = 8 * (c % (4 * KT));
    v8bf hi, lo;
#pragma unroll
    for (int e = 0; e < 8; ++e) hi[e] = lo[e] = (__bf16)0.f;
    if (k < p.rank) {
      const float* const h = p.h + ((int64_t)t.begin + r) * p.h_pitch + k;
      v4f v[8][2];      // all pieces' loads, then their sum in order
#pragma unroll
      for (int z = 0; z < 8; ++z)
        if (z < p.splits) {
          const float* const q = h + (int64_t)z * p.groups.R * p.h_pitch;
          v[z][0] = *reinterpret_cast<const v4f*>(q);
          v[z][1] = *reinterpret_cast<const v4f*>(q + 4);
        }
#pragma unroll
      for (int z = 1; z < 8; ++z)
        if (z < p.splits)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[0][0][e] += v[z][0][e];
            v[0][1][e] += v[z][1][e];
          }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = v[0][e / 4][e & 3] * scale;
        hi[e] = (__bf16)x;
        const float back = (float)hi[e];
        lo[e] = (__bf16)(fabsf(back) == __builtin_inff() ? 0.f : x - back);      // (inf - inf is no number)
      }
    }
    *reinterpret_cast<v8bf*>(parts + r * HP + k) = hi;
    *reinterpret_cast<v8bf*>(parts + r * HP + 32 * KT + k) = lo;
  }
}

// out += s B h, 64 columns a wave. MFMA: rows of B as its rows, places as its
// columns. The products pass through the wave's part of LDS, 16 places at a time,
// so that loads and stores of out cover whole stretches of a row, 16 bytes a lane
// whatever its alignment (a column a lane, for an odd stride, took 999x2115 16 us, so
// 10); a row's last columns, fewer than eight, go one by one. All old values are
// asked for before anything is multiplied.
template <int KT>
__global__ __launch_bounds__(256)
void lora_expand_kernel(LoraArgs p) {
  constexpr int PITCH = 68, HP = 64 * KT + 8;      // of a product's row (floats), of h's two parts (bf16)
  __shared__ __attribute__((aligned(16))) float lds[4 * 16 * PITCH];
  __shared__ __attribute__((aligned(16))) __bf16 parts[LORA_ROWS * HP];
  const groups::Tile t = groups::find_tile(p.groups, LORA_ROWS, p.parts, p.parts, groups::item_of(blockIdx.x, 1), false);
  if (t.rows <= 0) return;
  const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // rows of the tile, 8 at a time: lane / 8; all asked for at once
  int row[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int at = 16 * i + 8 * r + (lane >> 3);
      row[i][r] = p.groups.rows[t.begin + (at < t.rows ? at : 0)];
    }
  const int64_t n0 = (int64_t)t.part * LORA_COLS + 64 * wave;
  v4u b[KT][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int64_t n = n0 + 16 * i + col;
    n = n < p.N ? n : p.N - 1;         // columns past the last one are not kept
    const uint16_t* const row = p.b + (t.group * p.N + n) * p.rank;
#pragma unroll
    for (int s = 0; s < KT; ++s)       // (past the rank h is zero)
      b[s][i] = *reinterpret_cast<const v4u*>(row + (32 * s + 8 * g < p.rank ? 32 * s + 8 * g : 0));
  }
  split_h<KT>(p, t, parts);
  float* const mine = lds + wave * 16 * PITCH;
  // 8 columns a lane, of which `cols` there are
  const int c = 8 * (lane & 7), cols = p.N - n0 - c < 8 ? (int)(p.N - n0 - c) : 8;
  // Lanes with fewer ask for the row's last eight and keep `cols` of them; lanes
  // without a row or a column ask for others, and drop them.
  const int64_t at = cols == 8 ? n0 + c : p.N - 8;
  uint16_t* to[4][2];
  bool kept[4][2];
  v4u old[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int m = row[i][r];
      const bool is = m >= 0 && m < p.M;
      to[i][r] = p.out + (is ? m : 0) * p.ldo + at;
      kept[i][r] = is && cols > 0 && 16 * i + 8 * r + (lane >> 3) < t.rows;
    }
  if (p.N >= 8)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) old[i][r] = *reinterpret_cast<const groups::v4u_any*>(to[i][r]);
  // (LDS alone is waited for: the old values are still on their way)
  __builtin_amdgcn_s_waitcnt(WAITCNT_LGKM0);
  block_barrier();
  if (n0 >= p.N) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r0 = 16 * i;
    if (r0 >= t.rows) break;
    const __bf16* const h = parts + (r0 + col < t.rows ? r0 + col : 0) * HP + 8 * g;
    v4f acc[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < KT; ++s) {
      const v8bf hi = *reinterpret_cast<const v8bf*>(h + 32 * s), lo = *reinterpret_cast<const v8bf*>(h + 32 * (KT + s));
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand(b[s][q]), lo, acc[q], 0, 0, 0);
        acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand(b[s][q]), hi, acc[q], 0, 0, 0);
      }
    }
    asm volatile("" ::: "memory");   // the wave's own reads, its writes, its reads: in order
#pragma unroll
    for (int q = 0; q < 4; ++q) *reinterpret_cast<v4f*>(mine + col * PITCH + 16 * q + 4 * g) = acc[q];
    asm volatile("" ::: "memory");
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (!kept[i][r]) continue;
      const float* const from = mine + (8 * r + (lane >> 3)) * PITCH + c;
      const v4u o = old[i][r];
      if (cols == 8) {
        const v4f lo = *reinterpret_cast<const v4f*>(from), hi = *reinterpret_cast<const v4f*>(from + 4);
        v4u d;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = e < 2 ? lo[2 * e] : hi[2 * e - 4], y = e < 2 ? lo[2 * e + 1] : hi[2 * e - 3];
          d[e] = layer::pack_bf16(layer::bf16_lo(o[e]) + x, layer::bf16_hi(o[e]) + y);
        }
        *reinterpret_cast<groups::v4u_any*>(to[i][r]) = d;
      } else if (p.N >= 8) {
#pragma unroll
        for (int e = 1; e < 8; ++e)
          if (e >= 8 - cols) {
            const float x = e & 1 ? layer::bf16_hi(o[e / 2]) : layer::bf16_lo(o[e / 2]);
            to[i][r][e] = (uint16_t)layer::pack_bf16(x + from[e - (8 - cols)], 0.f);
          }
      } else {
        for (int e = 8 - cols; e < 8; ++e) to[i][r][e] = (uint16_t)layer::pack_bf16(layer::bf16_lo(to[i][r][e]) + from[e - (8 - cols)], 0.f);
      }
    }
  }
}

int64_t tiles_of(int64_t R, int32_t G, int rows) { return R / rows + (G < R ? G : R); }

// Places of the first launch's workgroups: 32 for larger ranks where the tiles are many,
// so that A comes from L2 half as often (us in all, 16 / 32: rank 64, 1536x7168, 4632
// tokens of 8 adapters 38.2 / 30.0, 2048 23.9 / 20.4, 1024 16.5 / 17.6, 64 of 32 10.2 /
// 11.5; rank 128, 4632 tokens 62.0 / 43.9; 8192x1536, rank 64, 4632 41.9 / 40.1, 2048 24.1 /
// 25.1).
int shrink_rows(int64_t R, int32_t G, int32_t rank) { return rank > 32 && tiles_of(R, G, 16) >= 128 ? 32 : 16; }

}  // namespace

// Pieces of K: enough that the first launch has 256 workgroups, of two steps a wave at
// least (us in all, 128 / 256 / 512 workgroups: 64 tokens of 32 adapters 8.1 / 7.6 / 7.8, 999
// of 20 18.3 / 16.8 / 17.9, 1024 of 4 15.5 / 13.3 / 14.4: the second launch reads every piece)
int lora_splits(int64_t R, int32_t G, int32_t rank, int64_t K) {
  const int64_t tiles = tiles_of(R, G, shrink_rows(R, G, rank)), steps = (K + 63) / 64;
  int64_t z = 256 / (tiles > 0 ? tiles : 1);
  if (z > steps / (2 * SHRINK_WAVES)) z = steps / (2 * SHRINK_WAVES);
  return z < 1 ? 1 : z > 8 ? 8 : (int)z;
}

int lora_pitch(int32_t rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

namespace {

int64_t shrink_workgroups(int64_t R, int32_t G, int32_t rank, int splits) {
  return (tiles_of(R, G, shrink_rows(R, G, rank)) * splits + 7) / 8 * 8;
}
int64_t expand_workgroups(int64_t R, int32_t G, int64_t N) { return (tiles_of(R, G, LORA_ROWS) * ((N + LORA_COLS - 1) / LORA_COLS) + 7) / 8 * 8; }

}  // namespace

int64_t lora_workgroups(int64_t R, int32_t G, int32_t rank, int64_t K, int64_t N) {
  const int64_t shrink = shrink_workgroups(R, G, rank, lora_splits(R, G, rank, K)), expand = expand_workgroups(R, G, N);
  return shrink > expand ? shrink : expand;
}

hipError_t launch_lora_add(LoraArgs p, hipStream_t stream) {
  p.h_pitch = lora_pitch(p.rank);
  p.parts = (int32_t)((p.N + LORA_COLS - 1) / LORA_COLS);
  const int64_t shrink = shrink_workgroups(p.groups.R, p.groups.G, p.rank, p.splits);
  const int64_t expand = expand_workgroups(p.groups.R, p.groups.G, p.N);
  // (16 places: LDS for two workgroups a CU up to rank 64)
  const bool wide = shrink_rows(p.groups.R, p.groups.G, p.rank) == 32;
  const auto first = p.h_pitch == 16   ? lora_shrink_kernel<1, 1, 4>
                     : p.h_pitch == 32 ? lora_shrink_kernel<1, 2, 3>
                     : p.h_pitch == 64 ? (wide ? lora_shrink_kernel<2, 4, 2> : lora_shrink_kernel<1, 4, 2>)
                                       : (wide ? lora_shrink_kernel<2, 8, 2> : lora_shrink_kernel<1, 8, 2>);
  hipLaunchKernelGGL(first, dim3((unsigned)shrink), dim3(64 * SHRINK_WAVES), 0, stream, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const auto second = p.rank <= 32 ? lora_expand_kernel<1> : p.rank <= 64 ? lora_expand_kernel<2> : lora_expand_kernel<4>;
  hipLaunchKernelGGL(second, dim3((unsigned)expand), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace iqp
