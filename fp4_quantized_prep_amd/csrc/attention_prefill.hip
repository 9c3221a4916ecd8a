// Attention of many query rows per sequence (prompts and their continuations)
// over the FP8 key/value cache: the formula of attention_decode.hip.
//
// Matrix-core bound: 4 D operations a visible (row, token) pair. A workgroup of
// four waves takes 128 rows (query heads of one key head by tokens, 32 a wave)
// and walks the visible tokens in units of 64:
//   * the unit's codes are loaded once (16 bytes a lane), widened once (keys
//     to bf16, values to fp16, both exact) and put in LDS, two units deep with one
//     barrier a unit, while the previous unit is computed;
//   * 32x32x16 MFMAs, tokens as the rows of the score product and dims as the
//     rows of the second one, query rows as columns of both. Score row
//     8 a + 4 h + b is token 16 (a / 2) + 8 h + 4 (a % 2) + b of its 32, so that
//     lane half h holds 8 consecutive tokens of each 16 and its scores are
//     already the second product's operand: probabilities never leave the lane;
//   * a unit's four 16-token granules lie in one block each, so block numbers,
//     scales and whether they are held are scalars. Key scales multiply the
//     scores, value exponents go into the probabilities' exponents (see
//     attention_decode.hip);
//   * 16-byte chunks in LDS are permuted by row (c ^ row % 16 in rows of 256
//     bytes, c ^ (row / 2) % 8 in rows of 128), so that the 16
//     lanes of a read cycle meet distinct banks.
// Workgroups are numbered with the key head fastest, so that with 8 heads an
// XCD's L2 holds one head's cache, longest row tiles first. Few rows against a
// long cache are split into Z pieces of the token range, joined by a second
// launch.
#include "attention_common.h"

namespace iqp {
namespace {

using namespace attn;

constexpr int PWAVES = 4;
constexpr int PROWS = 32 * PWAVES;     // rows of a workgroup
constexpr int SPLIT_GROUPS = 512;      // most workgroups of a split launch (partial results kept)

template <int D>
struct PartialTile {
  float m[PROWS], l[PROWS];
  float o[PROWS][D];
};

struct Work {
  int64_t begin, n, len;    // the sequence
  int64_t row0, rows;       // first row of the tile, rows of the sequence
  int64_t lo, hi;           // tokens that any row of the tile sees: [lo, hi)
  int s;
};

// Row tile `item` (numbering of find_sequence with 2^7 rows): false where there is none
__device__ __forceinline__ bool find_work(const AttnArgs& p, int64_t item, Work& w) {
  const SeqRows q = find_sequence(p.seq, item, p.group, 7, 1);
  w.s = q.s;
  w.begin = q.begin;
  w.n = q.end - q.begin;
  w.len = q.len;
  w.rows = w.n * p.group;
  if (w.n <= 0 || w.rows <= p.max_rows) return false;
  const int64_t tiles = (w.rows + PROWS - 1) / PROWS;
  const int64_t tile = item - item_key(q, p.group, 7, 1);
  if (tile >= tiles) return false;
  w.row0 = (tiles - 1 - tile) * PROWS;     // the longest first
  const int64_t last = w.row0 + PROWS < w.rows ? w.row0 + PROWS - 1 : w.rows - 1;
  const int64_t held = (int64_t)p.seq.max_blocks << p.seq.log_block;
  const int64_t first_pos = w.len - w.n + w.row0 / p.group, last_pos = w.len - w.n + last / p.group;
  w.lo = p.window > 0 && first_pos + 1 > p.window ? first_pos + 1 - p.window : 0;
  w.hi = last_pos + 1 < held ? last_pos + 1 : held;
  return true;
}

// largest of a lane's value and its partner's (lane ^ 32)
__device__ __forceinline__ float max_halves(float v) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float sum_halves(float v) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

template <int D>
struct Prefill {
  static constexpr int KS = D / 16;             // MFMA steps of a score
  static constexpr int DT = D / 32;             // output tiles
  static constexpr int LOADS = D / 64;          // 16-byte pieces of keys (and of values) a thread and unit
  static constexpr int K_BYTES = UNIT * D * 2, V_BYTES = D * UNIT * 2;
  static constexpr int LDS_BYTES = 2 * (K_BYTES + V_BYTES);

  // permutation of a key row's 16-byte chunks: rows of 256 bytes cover all
  // banks, rows of 128 half of them
  static __device__ __forceinline__ int key_swizzle(int tok) { return D == 128 ? tok & 15 : (tok >> 1) & 7; }

  struct Codes {
    v4u k[LOADS], v[LOADS];
  };
  // a unit's granules: lane's granule is lane % 4
  struct Granules {
    int blk;      // block number as the table has it (-1: past the table)
    int ks, vs;   // its scale bytes, turned into factors where they are used: a unit after their
                  // load, so that nothing waits for the codes loaded behind them
  };

  static __device__ __forceinline__ void run(const AttnArgs& p, int splits, uint8_t* lds) {
    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, col = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int head = (int)(blockIdx.x % (unsigned)p.Hk);
    const int64_t rest = blockIdx.x / (unsigned)p.Hk;
    const int z = (int)(rest % splits);
    Work w;
    if (!find_work(p, rest / splits, w)) return;

    const int64_t row = w.row0 + 32 * wave + col;
    const int64_t rc = row < w.rows ? row : w.rows - 1;
    const int64_t src = row_offset(w.begin, rc, head, p.group, D, p.ldq);
    v8bf fq[KS];
#pragma unroll
    for (int k = 0; k < KS; ++k) fq[k] = *reinterpret_cast<const v8bf*>(p.q + src + 16 * k + 8 * half);
    // tokens relative to the unit range's first, 32 bits wide
    const int64_t u_lo = w.lo / UNIT, u_hi = w.hi > w.lo ? (w.hi + UNIT - 1) / UNIT : u_lo;
    const int64_t u0 = u_lo + (u_hi - u_lo) * z / splits, u1 = u_lo + (u_hi - u_lo) * (z + 1) / splits;
    const int64_t base = u0 * UNIT;
    const int units = (int)(u1 - u0);
    const int64_t pos = w.len - w.n + rc / p.group;
    const int see_hi = (int)(pos + 1 - base < -1 ? -1 : pos + 1 - base);
    const int64_t lo64 = p.window > 0 ? pos + 1 - p.window - base : -1;
    const int see_lo = (int)(lo64 < -1 ? -1 : lo64);
    // of the wave's columns: what all of them see, and the last token any of them sees
    const int64_t wr0 = w.row0 + 32 * wave < w.rows ? w.row0 + 32 * wave : w.rows - 1;
    const int64_t wr1 = wr0 + 31 < w.rows ? wr0 + 31 : w.rows - 1;
    const int64_t p0 = w.len - w.n + wr0 / p.group - base, p1 = w.len - w.n + wr1 / p.group - base;
    const int all_hi = (int)(p0 + 1 < -1 ? -1 : p0 + 1), any_hi = (int)(p1 + 1 < -1 ? -1 : p1 + 1);
    const int64_t al = p.window > 0 ? p1 + 1 - p.window : -1, an = p.window > 0 ? p0 + 1 - p.window : -1;
    const int all_lo = (int)(al < -1 ? -1 : al), any_lo = (int)(an < -1 ? -1 : an);
    const bool idle = w.row0 + 32 * wave >= w.rows;      // no rows at all

    const int32_t* const table = p.seq.table + (int64_t)w.s * p.seq.ld_table;
    const int lb = p.seq.log_block, inside = (1 << lb) - 1;
    const int gr = lane & 3;

    auto load_block = [&](int u) __attribute__((always_inline)) {
      const int64_t b = (base + (int64_t)u * UNIT + 16 * gr) >> lb;
      return u < units && b < p.seq.max_blocks ? table[b] : -1;
    };
    auto held_block = [&](int blk) __attribute__((always_inline)) { return blk >= 0 && blk < p.seq.n_blocks; };
    auto load_granules = [&](int blk) __attribute__((always_inline)) {
      Granules g;
      g.blk = blk;
      const int64_t at = (int64_t)(held_block(blk) ? blk : 0) * p.Hk + head;
      g.ks = p.k_scales[at];
      g.vs = p.v_scales[at];
      return g;
    };
    // the thread's codes of unit u, whose blocks are in blk
    auto load_codes = [&](int u, int blk) __attribute__((always_inline)) {
      Codes c;
      const int64_t t0 = base + (int64_t)u * UNIT;
      const int own = held_block(blk) ? blk : 0;
      const uint8_t* vb = p.v_cache + ((((int64_t)own * p.Hk + head) * D) << lb) + ((t0 + 16 * gr) & inside);
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        // keys: 16 dims of a token; a wave's tokens lie in one granule
        constexpr int PIECES = D / 16;
        const int x = tid + 256 * i;
        const int tok = x / PIECES, piece = x % PIECES;
        const int granule = (64 * wave + 256 * i) / PIECES / 16;
        const int kb = __builtin_amdgcn_readlane(own, granule);
        const uint8_t* ks = p.k_cache + (((int64_t)kb * p.Hk + head) << lb) * D + ((t0 + tok) & inside) * D + 16 * piece;
        c.k[i] = *reinterpret_cast<const v4u*>(ks);
        // values: 16 tokens of dim x / 4
        c.v[i] = *reinterpret_cast<const v4u*>(vb + ((int64_t)(x >> 2) << lb));
      }
      return c;
    };
    auto store_codes = [&](int u, const Codes& c, bool held) __attribute__((always_inline)) {
      uint8_t* const kl = lds + (u & 1) * (K_BYTES + V_BYTES);
      uint8_t* const vl = kl + K_BYTES;
      const int64_t t0 = base + (int64_t)u * UNIT + 16 * gr;
      const int64_t hi64 = w.len - t0, lo64v = w.lo - t0;
      const int hi = held ? (hi64 > 16 ? 16 : (int)hi64) : 0, lo = lo64v > 16 ? 16 : (int)(lo64v < 0 ? 0 : lo64v);
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        constexpr int PIECES = D / 16;
        const int x = tid + 256 * i;
        const int tok = x / PIECES, piece = x % PIECES;
        uint8_t* const kr = kl + tok * (2 * D);
        *reinterpret_cast<v8bf*>(kr + 16 * ((2 * piece) ^ key_swizzle(tok))) = widen_bf16(c.k[i][0], c.k[i][1]);
        *reinterpret_cast<v8bf*>(kr + 16 * ((2 * piece + 1) ^ key_swizzle(tok))) = widen_bf16(c.k[i][2], c.k[i][3]);
        v4u v = c.v[i];
        // behind the sequence, before the window or not held: must not reach
        // the product (0 * NaN)
        if (lo > 0 || hi < 16) v = clear_outside(v, lo, hi);
        const int d = x >> 2;
        uint8_t* const vr = vl + d * (2 * UNIT);
        *reinterpret_cast<v8h*>(vr + 16 * ((2 * gr) ^ ((d >> 1) & 7))) = widen_f16(v[0], v[1]);
        *reinterpret_cast<v8h*>(vr + 16 * ((2 * gr + 1) ^ ((d >> 1) & 7))) = widen_f16(v[2], v[3]);
      }
    };

    float m = LOWEST, l = 0.f;
    v16f o[DT];
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[t][r] = 0.f;

    // the key row of score row `col`, and the swizzle of the lane's operand reads
    const int krow = 16 * (col >> 4) + 8 * ((col >> 2) & 1) + 4 * ((col >> 3) & 1) + (col & 3);
    if (units > 0) {
      int blk = load_block(0), blk_next = load_block(1);
      Granules gn = load_granules(blk);
      {
        const Codes c = load_codes(0, blk);
        store_codes(0, c, held_block(blk));
      }
      __syncthreads();
      for (int u = 0; u < units; ++u) {
        const Granules g = gn;
        Codes next;
        const int blk1 = blk_next;
        if (u + 1 < units) {
          blk_next = load_block(u + 2);
          gn = load_granules(blk1);
          next = load_codes(u + 1, blk1);
        }
        const int t0 = u * UNIT;
        if (!idle && t0 < any_hi && t0 + UNIT > any_lo) {
          const uint8_t* const kl = lds + (u & 1) * (K_BYTES + V_BYTES);
          const uint8_t* const vl = kl + K_BYTES;
          v16f sc[2];
#pragma unroll
          for (int a = 0; a < 2; ++a) {
#pragma unroll
            for (int r = 0; r < 16; ++r) sc[a][r] = 0.f;
            const uint8_t* const kr = kl + (32 * a + krow) * (2 * D);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              const v8bf fk = *reinterpret_cast<const v8bf*>(kr + 16 * ((2 * k + half) ^ key_swizzle(krow)));
              sc[a] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fk, fq[k], sc[a], 0, 0, 0);
            }
          }
          // granule 2 a + (r >> 3): scalars
          float kmul[4], ve[4], vinv[4];
          bool in[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int kb = __builtin_amdgcn_readlane(g.ks, i), vb = __builtin_amdgcn_readlane(g.vs, i);
            kmul[i] = p.scale_log2 * pow2(max(kb - 127, -126));
            ve[i] = (float)(vb - 127);
            vinv[i] = pow2(min(127 - vb, 127));
            in[i] = held_block(__builtin_amdgcn_readlane(g.blk, i));
          }
          if (t0 + UNIT > all_hi || t0 < all_lo || !(in[0] && in[1] && in[2] && in[3])) {
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
              for (int r = 0; r < 16; ++r) {
                const int i = 2 * a + (r >> 3);
                const int tok = t0 + 32 * a + 16 * (r >> 3) + 8 * half + (r & 7);
                sc[a][r] = in[i] && tok >= see_lo && tok < see_hi ? sc[a][r] * kmul[i] + ve[i] : -INFINITY;
              }
          } else {
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
              for (int r = 0; r < 16; ++r) sc[a][r] = sc[a][r] * kmul[2 * a + (r >> 3)] + ve[2 * a + (r >> 3)];
          }
          float mx = sc[0][0];
#pragma unroll
          for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int r = 0; r < 16; ++r) mx = fmaxf(mx, sc[a][r]);
          mx = fmaxf(m, max_halves(mx));
          if (__ballot(mx > m) != 0) {     // some column's maximum rose: rescale
            const float alpha = __builtin_amdgcn_exp2f(m - mx);
            m = mx;
            l *= alpha;
#pragma unroll
            for (int t = 0; t < DT; ++t)
#pragma unroll
              for (int r = 0; r < 16; ++r) o[t][r] *= alpha;
          }
          v8h fp[2][2];
#pragma unroll
          for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              float x[8], sum = 0.f;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                x[j] = __builtin_amdgcn_exp2f(sc[a][8 * s + j] - m);
                sum += x[j];
              }
              l += sum * vinv[2 * a + s];
              fp[a][s] = v8h{(_Float16)x[0], (_Float16)x[1], (_Float16)x[2], (_Float16)x[3],
                             (_Float16)x[4], (_Float16)x[5], (_Float16)x[6], (_Float16)x[7]};
            }
#pragma unroll
          for (int t = 0; t < DT; ++t) {
            const int d = 32 * t + col;
            const uint8_t* const vr = vl + d * (2 * UNIT);
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
              for (int s = 0; s < 2; ++s) {
                const v8h fv = *reinterpret_cast<const v8h*>(vr + 16 * ((4 * a + 2 * s + half) ^ ((d >> 1) & 7)));
                o[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fv, fp[a][s], o[t], 0, 0, 0);
              }
          }
        }
        if (u + 1 < units) store_codes(u + 1, next, held_block(blk1));
        __syncthreads();   // unit u + 1 is in LDS; unit u is read by every wave
      }
    }

    l = sum_halves(l);
    if (row >= w.rows) return;
    if (splits == 1) {
      const float inv = inverse_sum(l);
      uint16_t* const dst = p.out + row_offset(w.begin, row, head, p.group, D, p.ldo) + 4 * half;
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int a = 0; a < 4; ++a)
          *reinterpret_cast<v2u*>(dst + 32 * t + 8 * a) =
              v2u{pack_bf16(o[t][4 * a] * inv, o[t][4 * a + 1] * inv), pack_bf16(o[t][4 * a + 2] * inv, o[t][4 * a + 3] * inv)};
    } else {
      PartialTile<D>& part = reinterpret_cast<PartialTile<D>*>(p.workspace)[blockIdx.x];
      const int r0 = 32 * wave + col;
      if (half == 0) {
        part.m[r0] = m;
        part.l[r0] = l;
      }
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int a = 0; a < 4; ++a)
          *reinterpret_cast<v4f*>(&part.o[r0][32 * t + 8 * a + 4 * half]) =
              v4f{o[t][4 * a], o[t][4 * a + 1], o[t][4 * a + 2], o[t][4 * a + 3]};
    }
  }
};

template <int D>
__global__ __launch_bounds__(PWAVES * 64, 2)
void attention_prefill_kernel(AttnArgs p, int splits) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[Prefill<D>::LDS_BYTES];
  Prefill<D>::run(p, splits, lds);
}

// Joins the pieces of a split launch: a workgroup per row tile, key head and 16 rows
template <int D>
__global__ __launch_bounds__(256)
void attention_prefill_join_kernel(AttnArgs p, int splits) {
  const int64_t item = blockIdx.x / (unsigned)p.Hk;
  const int head = (int)(blockIdx.x % (unsigned)p.Hk);
  Work w;
  if (!find_work(p, item, w)) return;
  const PartialTile<D>* const parts = reinterpret_cast<const PartialTile<D>*>(p.workspace);
  for (int i = threadIdx.x; i < 16 * (D / 4); i += 256) {
    const int r = 16 * blockIdx.y + i / (D / 4), d = 4 * (i % (D / 4));
    if (w.row0 + r >= w.rows) break;
    float mx = LOWEST;
    for (int z = 0; z < splits; ++z) mx = fmaxf(mx, parts[(item * splits + z) * p.Hk + head].m[r]);
    float sum = 0.f;
    v4f acc = {0.f, 0.f, 0.f, 0.f};
    for (int z = 0; z < splits; ++z) {
      const PartialTile<D>& x = parts[(item * splits + z) * p.Hk + head];
      const float a = __builtin_amdgcn_exp2f(x.m[r] - mx);
      sum += x.l[r] * a;
      const v4f v = *reinterpret_cast<const v4f*>(&x.o[r][d]);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] += v[j] * a;
    }
    const float inv = inverse_sum(sum);
    uint16_t* const dst = p.out + row_offset(w.begin, w.row0 + r, head, p.group, D, p.ldo) + d;
    *reinterpret_cast<v2u*>(dst) = v2u{pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv)};
  }
}

template <int D>
hipError_t launch(const AttnArgs& p, hipStream_t stream) {
  const int64_t items = ((p.seq.T * p.group) >> 7) + p.seq.S, pairs = items * p.Hk;
  // split where the row tiles leave CUs idle and the table allows for pieces of
  // at least four units
  const int64_t longest = ((int64_t)p.seq.max_blocks << p.seq.log_block) / (4 * UNIT);
  int64_t splits = SPLIT_GROUPS / pairs;
  if (splits > longest) splits = longest;
  if (splits < 1) splits = 1;
  if (pairs * splits > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL((attention_prefill_kernel<D>), dim3((unsigned)(pairs * splits)), dim3(PWAVES * 64), 0, stream, p, (int)splits);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  hipLaunchKernelGGL((attention_prefill_join_kernel<D>), dim3((unsigned)pairs, PROWS / 16), dim3(256), 0, stream, p, (int)splits);
  return hipGetLastError();
}

}  // namespace

int64_t attention_prefill_workspace_bytes(int D) {
  return (int64_t)SPLIT_GROUPS * (D == 64 ? sizeof(PartialTile<64>) : sizeof(PartialTile<128>));
}

hipError_t launch_attention_prefill(const AttnArgs& p, int D, hipStream_t stream) {
  return D == 64 ? launch<64>(p, stream) : launch<128>(p, stream);
}

}  // namespace iqp
