// Attention of many query rows per sequence (prompts and their continuations)
// over the FP8 key/value cache: the formula of attention_decode.hip.
//
// Bound by the matrix cores and the vector instructions of the softmax
// together: 4 D operations a visible (row, token) pair on the former, seven to eight
// instructions on the latter (four to five of them the softmax, the others widening and
// addresses), which take as long at D 128 and twice as long at D 64. A workgroup's four waves take 128 rows (query heads of one key head by
// tokens, 32 a wave) and walk the visible tokens in units of 64:
//   * a unit's codes are loaded once (16 bytes a lane) two units ahead, widened
//     once (keys to bf16, values to fp16, both exact) and put in LDS beside the
//     score MFMAs of the unit before; one barrier a unit;
//   * 32x32x16 MFMAs, tokens as the rows of the score product and dims as the
//     rows of the second one, query rows as columns of both. Score row
//     8 a + 4 h + b is token 16 (a / 2) + 8 h + 4 (a % 2) + b of its 32, so that
//     lane half h holds 8 consecutive tokens of each 16 and its scores are
//     already the second product's operand: probabilities never leave the lane.
//     The weights of 16 tokens are computed beside the second product of the 16
//     before;
//   * a unit's four 16-token granules lie in one block each, so block numbers,
//     scales and whether they are held are scalars. Key scales multiply the
//     scores, value exponents go into the probabilities' exponents (see
//     attention_decode.hip);
//   * a tile of few rows (a single token beside prompts, the rest of a prompt) is
//     computed as the decode kernel computes it, and so are rows of very large scores;
//   * 16-byte chunks in LDS are permuted by row, so that the lanes of a cycle
//     meet distinct banks.
// Workgroups are numbered with the key head fastest, so that with 8 heads an
// XCD's L2 holds one head's cache, longest row tiles first. Where there are few,
// SETS = 2 gives a workgroup eight waves, of which four take the first half of
// the tokens and four the second, joined in LDS; where there are very few, the
// token range is split into Z pieces, joined by a second launch.
//
// Measured: 4632 tokens, 64 heads of 128 over 8: 380 us, 0.92 PFLOP/s (MFMAs alone
// 190 us of it; a large bf16 product of the library reaches 1.39).
#include <type_traits>

#include "attention_rows.h"

namespace iqp {
namespace {

using namespace attn;

constexpr int PWAVES = 4;
constexpr int PROWS = 32 * PWAVES;     // rows of a workgroup
// A tile of no more rows than this goes to FewRows, whose waves share out the tokens
// and not the rows (24 sequences of 1 to 30 tokens, 8 heads over 1, after up to 3900:
// 69 us; with 64 instead 106)
constexpr int FEW_ROWS = 32;
constexpr float SLACK = 8.f;
constexpr float LARGE = 8388608.f;     // 2^23, where float32 steps are 1
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
  if (tile < 0 || tile >= tiles) return false;
  w.row0 = (tiles - 1 - tile) * PROWS;     // the longest first
  const int64_t last = w.row0 + PROWS < w.rows ? w.row0 + PROWS - 1 : w.rows - 1;
  const int64_t held = (int64_t)p.seq.max_blocks << p.seq.log_block;
  const int64_t first_pos = w.len - w.n + w.row0 / p.group, last_pos = w.len - w.n + last / p.group;
  w.lo = p.window > 0 && first_pos + 1 > p.window ? first_pos + 1 - p.window : 0;
  w.hi = last_pos + 1 < held ? last_pos + 1 : held;
  return true;
}

// bits 0 .. n - 1, none below 0, all from 32 on
__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? ~0u : (1u << (n < 0 ? 0 : n)) - 1u; }

// The largest of three in one instruction, v_maximum3_f32 (for fmaxf the compiler would
// quiet each operand first). Not inline asm: operands are MFMA results, and the
// compiler counts the wait states behind an MFMA only to instructions of its own.
// A NaN is kept; it makes its row NaN in any case.
__device__ __forceinline__ float max3(float a, float b, float c) {
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
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

template <int D, int SETS>
struct Prefill {
  static constexpr int U = UNIT, GR = U / 16;   // tokens of a unit, its granules
  static constexpr int KS = D / 16;             // MFMA steps of a score
  static constexpr int NA = U / 32;             // score tiles
  static constexpr int LOADS = D / 64;          // 16-byte pieces of keys (and of values) a thread and unit
  static constexpr int DT = D / 32;             // output tiles
  static constexpr int K_BYTES = U * D * 2, V_BYTES = D * U * 2;
  static constexpr int SET_BYTES = 2 * (K_BYTES + V_BYTES), LDS_BYTES = SETS * SET_BYTES;
  static constexpr int FLAG_BYTES = 4 * SETS * PROWS;   // LDS's last: whether a row met a large score

  // Where 16-byte chunk c of a key row, of a value row lies in it. A read takes one
  // chunk of 16 rows, which then lie in distinct banks of 64; a store every second
  // chunk of one row (256 bytes) or of two (128), distinct among 32.
  static __device__ __forceinline__ int narrow_chunk(int row, int c) { return c ^ ((row >> 1) & 7) ^ (row & 1); }
  static __device__ __forceinline__ int key_chunk(int tok, int c) { return D == 128 ? c ^ (c >> 3) ^ (tok & 15) : narrow_chunk(tok, c); }
  static __device__ __forceinline__ int value_chunk(int dim, int c) { return narrow_chunk(dim, c); }

  struct Codes {
    v4u k[LOADS], v[LOADS];
  };
  // a unit's granules: lane's granule is lane % GR
  struct Granules {
    int blk;      // block number as the table has it (-1: past the table)
    int ks, vs;   // its scale bytes, turned into factors where they are used: a unit after their
                  // load, so that nothing waits for the codes loaded behind them
  };

  // whether each row of the tile met a large score, in each set of waves
  static __device__ __forceinline__ int* large_flags(uint8_t* lds_all) { return reinterpret_cast<int*>(lds_all + LDS_BYTES - FLAG_BYTES); }
  static __device__ __forceinline__ bool is_large(const int* flags, int row) {
    return (SETS == 1 ? flags[row] : flags[row] | flags[PROWS + row]) != 0;
  }

  // The tile's rows, or those that are large alone, as the decode kernel computes them
  template <bool LARGE_ONLY>
  static __device__ __forceinline__ void few_rows(const AttnArgs& p, int splits, uint8_t* lds_all, const Work& w, int head, int z,
                                                  int64_t u_lo, int64_t u_hi) {
    using Few = FewRows<D, 1, SETS * PWAVES>;
    static_assert(sizeof(typename Few::Lds) <= LDS_BYTES - FLAG_BYTES, "in the units' place");
    PartialTile<D>& part = reinterpret_cast<PartialTile<D>*>(p.workspace)[blockIdx.x];
    const SeqRows seq = {w.s, (int)w.begin, (int)(w.begin + w.n), (int)w.len};
    const int64_t u0 = u_lo + (u_hi - u_lo) * z / splits, u1 = u_lo + (u_hi - u_lo) * (z + 1) / splits;
    const int64_t end = w.row0 + PROWS < w.rows ? w.row0 + PROWS : w.rows;
    const int* const flags = large_flags(lds_all);
    for (int64_t r0 = w.row0; r0 < end; r0 += Few::ROWS) {
      const int at = (int)(r0 - w.row0);
      if (LARGE_ONLY && __ballot(is_large(flags, at + (threadIdx.x & (Few::ROWS - 1)))) == 0) continue;
      Few::run(p, seq, r0, head, u0, u1 - u0, *reinterpret_cast<typename Few::Lds*>(lds_all),
               [&](int r, int d, float mx, float sum, v4f acc) __attribute__((always_inline)) {
        if (LARGE_ONLY && !is_large(flags, at + r)) return;
        if (splits == 1) {
          const float inv = inverse_sum(sum);
          uint16_t* const dst = p.out + row_offset(w.begin, r0 + r, head, p.group, D, p.ldo) + d;
          *reinterpret_cast<v2u*>(dst) = v2u{pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv)};
        } else {
          const int i = at + r;
          *reinterpret_cast<v4f*>(&part.o[i][d]) = acc;
          if (d == 0) {
            part.m[i] = mx;
            part.l[i] = sum;
          }
        }
      });
      __syncthreads();
    }
  }

  // The tile's rows on 32x32 MFMAs. Whether some of them, not written then, have scores
  // too large for that (below): LDS holds which ones.
  static __device__ __forceinline__ bool many_rows(const AttnArgs& p, int splits, uint8_t* lds_all, const Work& w, int head, int z,
                                                   int64_t u_lo, int64_t u_hi) {
    const int tid = threadIdx.x % (64 * PWAVES), lane = tid & 63, half = lane >> 5, col = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int set = SETS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / (64 * PWAVES));
    uint8_t* const lds = lds_all + set * SET_BYTES;

    const int64_t row = w.row0 + 32 * wave + col;
    const int64_t rc = row < w.rows ? row : w.rows - 1;
    const int64_t src = row_offset(w.begin, rc, head, p.group, D, p.ldq);
    v8bf fq[KS];
#pragma unroll
    for (int k = 0; k < KS; ++k) fq[k] = *reinterpret_cast<const v8bf*>(p.q + src + 16 * k + 8 * half);
    // tokens relative to the unit range's first, 32 bits wide
    const int64_t cuts = (int64_t)SETS * splits, cut = (int64_t)SETS * z + set;
    const int64_t u0 = u_lo + (u_hi - u_lo) * cut / cuts, u1 = u_lo + (u_hi - u_lo) * (cut + 1) / cuts;
    const int64_t base = u0 * U;
    const int units = (int)(u1 - u0);
    // rounds of the workgroup: a set with a unit less computes one of which nothing is held
    const int turns = SETS == 1 ? units : (int)((u_hi - u_lo + cuts - 1) / cuts);
    const int64_t pos = w.len - w.n + rc / p.group;
    const int see_hi = (int)(pos + 1 - base < -1 ? -1 : pos + 1 - base);
    const int64_t lo64 = p.window > 0 ? pos + 1 - p.window - base : -1;
    const int see_lo = (int)(lo64 < -1 ? -1 : lo64);
    // what all of the wave's columns see
    const int64_t wr0 = w.row0 + 32 * wave < w.rows ? w.row0 + 32 * wave : w.rows - 1;
    const int64_t wr1 = wr0 + 31 < w.rows ? wr0 + 31 : w.rows - 1;
    const int64_t p0 = w.len - w.n + wr0 / p.group - base, p1 = w.len - w.n + wr1 / p.group - base;
    const int all_hi = (int)(p0 + 1 < -1 ? -1 : p0 + 1);
    const int64_t al = p.window > 0 ? p1 + 1 - p.window : -1;
    const int all_lo = (int)(al < -1 ? -1 : al);

    const int32_t* const table = p.seq.table + (int64_t)w.s * p.seq.ld_table;
    const int lb = p.seq.log_block, inside = (1 << lb) - 1;
    const int gr = lane & (GR - 1);

    auto load_block = [&](int u) __attribute__((always_inline)) {
      const int64_t b = (base + (int64_t)u * U + 16 * gr) >> lb;
      return u < units && b < p.seq.max_blocks ? table[b] : -1;
    };
    auto held_block = [&](int blk) __attribute__((always_inline)) { return (unsigned)blk < (unsigned)p.seq.n_blocks; };
    auto load_granules = [&](int blk) __attribute__((always_inline)) {
      Granules g;
      g.blk = blk;
      const int64_t at = (int64_t)(held_block(blk) ? blk : 0) * p.Hk + head;
      g.ks = p.k_scales[at];
      g.vs = p.v_scales[at];
      return g;
    };
    // the thread's codes of unit u, whose blocks are in blk. Keys: 16 dims of
    // token tok + 256 i / PIECES; a wave's tokens lie in one granule, so the block
    // is a scalar. (Units start at multiples of U: the token within its block is
    // the sum of the unit's and the thread's.) Values: 16 tokens of a dim.
    constexpr int PIECES = D / 16, KSTEP = 256 / PIECES, VSTEP = 256 / GR;   // rows between a thread's pieces
    const int tok = tid / PIECES, piece = tid % PIECES, dim = tid / GR;
    unsigned key_at[LOADS], value_at[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      key_at[i] = (unsigned)(((tok + KSTEP * i) & inside) * D + 16 * piece);
      value_at[i] = (unsigned)(((dim + VSTEP * i) << lb) + ((16 * gr) & inside));
    }
    auto load_codes = [&](int u, int blk) __attribute__((always_inline)) {
      Codes c;
      const int t0 = (int)(base + (int64_t)u * U) & inside;
      const unsigned own = held_block(blk) ? blk : 0;
      const uint8_t* const vb = p.v_cache + ((((uint64_t)own * (unsigned)p.Hk + head) * D) << lb) + t0;
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const unsigned kb = __builtin_amdgcn_readlane(own, (64 * wave / PIECES + KSTEP * i) / 16);
        c.k[i] = *reinterpret_cast<const v4u*>(p.k_cache + ((((uint64_t)kb * (unsigned)p.Hk + head) << lb) + t0) * D + key_at[i]);
        c.v[i] = *reinterpret_cast<const v4u*>(vb + value_at[i]);
      }
      return c;
    };
    const int key_to = tok * (2 * D), value_to = K_BYTES + dim * (2 * U);
    const int key_to0 = key_to + 16 * key_chunk(tok, 2 * piece), key_to1 = key_to + 16 * key_chunk(tok, 2 * piece + 1);
    const int value_to0 = value_to + 16 * value_chunk(dim, 2 * gr), value_to1 = value_to + 16 * value_chunk(dim, 2 * gr + 1);
    // values behind the sequence, before the window or not held must not reach
    // the product (0 * NaN)
    auto clear_codes = [&](int u, Codes& c, int blk) __attribute__((always_inline)) {
      const int64_t t0 = base + (int64_t)u * U;
      if (t0 < w.lo || t0 + U > w.len || __ballot(!held_block(blk)) != 0) {
        const int64_t hi64 = w.len - t0 - 16 * gr, lo64 = w.lo - t0 - 16 * gr;
        const int hi = held_block(blk) ? (hi64 > 16 ? 16 : (int)hi64) : 0, lo = lo64 > 16 ? 16 : (int)(lo64 < 0 ? 0 : lo64);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) c.v[i] = clear_outside(c.v[i], lo, hi);
      }
    };
    // piece j (0 .. 4 LOADS - 1) of the thread's codes to buffer BUF, widened
    // (KSTEP and VSTEP rows on, the swizzles are the same)
    auto store_codes = [&](const Codes& c, int j, auto buf) __attribute__((always_inline)) {
      constexpr int BUF = decltype(buf)::value * (K_BYTES + V_BYTES);
      const int i = j >> 2;
      if ((j & 3) == 0) *reinterpret_cast<v8bf*>(lds + key_to0 + (BUF + KSTEP * i * 2 * D)) = widen_bf16(c.k[i][0], c.k[i][1]);
      if ((j & 3) == 1) *reinterpret_cast<v8bf*>(lds + key_to1 + (BUF + KSTEP * i * 2 * D)) = widen_bf16(c.k[i][2], c.k[i][3]);
      if ((j & 3) == 2) *reinterpret_cast<v8h*>(lds + value_to0 + (BUF + VSTEP * i * 2 * U)) = widen_f16(c.v[i][0], c.v[i][1]);
      if ((j & 3) == 3) *reinterpret_cast<v8h*>(lds + value_to1 + (BUF + VSTEP * i * 2 * U)) = widen_f16(c.v[i][2], c.v[i][3]);
    };

    float m = LOWEST, l = 0.f;
    bool large = false;
    v16f o[DT];
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[t][r] = 0.f;

    // the key row of score row `col`; operand reads: a lane's offsets within a
    // buffer, everything else an immediate
    const int krow = 16 * (col >> 4) + 8 * ((col >> 2) & 1) + 4 * ((col >> 3) & 1) + (col & 3);
    int koff[KS], voff[GR];
#pragma unroll
    for (int k = 0; k < KS; ++k) koff[k] = krow * (2 * D) + 16 * key_chunk(krow, 2 * k + half);
#pragma unroll
    for (int i = 0; i < GR; ++i) voff[i] = K_BYTES + col * (2 * U) + 16 * value_chunk(col, 2 * i + half);
    // a unit's granules in scalar registers (so no floating-point values);
    // granule 2 a + (r >> 3) holds score register r of tile a
    struct Scales {
      int kmul[GR];   // bits of scale * log2(e) * 2^(key exponent)
      int vb[GR];     // value scale byte
      int held;       // bit i: granule i is held
    };
    const int scale_bits = __builtin_amdgcn_readfirstlane(__float_as_int(p.scale_log2));
    auto scales_of = [&](const Granules& g) __attribute__((always_inline)) {
      Scales s;
      s.held = 0;
#pragma unroll
      for (int i = 0; i < GR; ++i) {
        // never 0, so that a masked score stays -inf: below 2^-100 every score is 0 to float32's last bit
        const int e = (scale_bits >> 23) + __builtin_amdgcn_readlane(g.ks, i) - 127;
        s.kmul[i] = (scale_bits & 0x7FFFFF) | (min(max(e, 27), 254) << 23);
        s.vb[i] = __builtin_amdgcn_readlane(g.vs, i);
        s.held |= held_block(__builtin_amdgcn_readlane(g.blk, i)) ? 1 << i : 0;
      }
      return s;
    };
    auto exponent_of = [&](const Scales& s, int i) __attribute__((always_inline)) { return (float)(s.vb[i] - 127); };
    auto kmul_of = [&](const Scales& s, int i) __attribute__((always_inline)) { return __int_as_float(s.kmul[i]); };
    auto vinv_of = [&](const Scales& s, int i) __attribute__((always_inline)) { return __int_as_float(max(254 - s.vb[i], 1) << 23); };

    // unit u, whose codes are in buffer BUF of LDS; beside the score MFMAs the
    // next unit's codes go to the other buffer, then the one's after it are loaded
    auto compute = [&](int u, const Scales& g, const Codes& next, auto buf, auto load) __attribute__((always_inline)) {
      using Other = std::integral_constant<int, 1 - decltype(buf)::value>;
      constexpr int BUF = decltype(buf)::value * (K_BYTES + V_BYTES);
      const int t0 = u * U;
      // operands are read AHEAD MFMAs before their use
      constexpr int AHEAD = 3, NQK = NA * KS, NPV = GR * DT;
      auto key = [&](int j) __attribute__((always_inline)) {      // j = NA k + a
        return *reinterpret_cast<const v8bf*>(lds + koff[j / NA] + (BUF + 32 * (j % NA) * 2 * D));
      };
      auto value = [&](int j) __attribute__((always_inline)) {    // j = DT i + t
        return *reinterpret_cast<const v8h*>(lds + voff[j / DT] + (BUF + 32 * (j % DT) * 2 * U));
      };
      v16f sc[NA];
      v8bf fk[NQK];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) fk[j] = key(j);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < NQK; ++j) {
        const v16f zero = {};
        sc[j % NA] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fk[j], fq[j / NA], j < NA ? zero : sc[j % NA], 0, 0, 0);
        if (j + AHEAD < NQK) fk[j + AHEAD] = key(j + AHEAD);
#pragma unroll
        for (int e = 4 * LOADS * j / NQK; e < 4 * LOADS * (j + 1) / NQK; ++e) store_codes(next, e, Other{});
        __builtin_amdgcn_sched_barrier(0);
      }
      load();
      __builtin_amdgcn_sched_barrier(0);
      if (t0 + U > all_hi || t0 < all_lo || g.held != (1 << GR) - 1) {
        // a bit a token: those of the unit that the row sees, the lane's 8 of each
        // granule, the held granules'; then two instructions a score
        const uint32_t w0 = below(see_hi - t0) & ~below(see_lo - t0), w1 = below(see_hi - t0 - 32) & ~below(see_lo - t0 - 32);
        const uint32_t bits = __builtin_amdgcn_perm(w1, w0, 0x06040200u + 0x01010101u * half) &
                              (((uint32_t)g.held * 0x00204081u & 0x01010101u) * 255u);
#pragma unroll
        for (int a = 0; a < NA; ++a)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const uint32_t sees = (uint32_t)((int)(bits << (31 - (16 * a + r))) >> 31);
            sc[a][r] = __uint_as_float((sees & __float_as_uint(sc[a][r])) | (~sees & 0xFF800000u));   // or -inf
          }
      }
      // the maximum, granule by granule (one factor each)
      float mx = LOWEST;
#pragma unroll
      for (int i = 0; i < GR; ++i) {
        const v16f& x = sc[i >> 1];
        const int r = 8 * (i & 1);
        const float gm = max3(max3(x[r], x[r + 1], x[r + 2]), max3(x[r + 3], x[r + 4], x[r + 5]), max3(x[r + 6], x[r + 7], x[r + 7]));
        mx = fmaxf(mx, __builtin_fmaf(gm, kmul_of(g, i), exponent_of(g, i)));
      }
      mx = max_halves(mx);
      // m follows the maximum only where it rose by more than SLACK (log2):
      // what is summed is then seldom rescaled, and weights, computed times
      // 2^(FP16_TOP - SLACK), stay below 2^FP16_TOP. Those that fp16 holds as
      // subnormals, below 2^-21 of the largest, are off by at most 2^-32 of it
      if (__ballot(mx > m + SLACK) != 0) {
        const float mn = fmaxf(m, mx), alpha = __builtin_amdgcn_exp2f(m - mn);
        // A weight's exponent takes score, factor and maximum in one rounding, but the
        // maximum was rounded before: off by half its step, which from LARGE on could put
        // all of the row's weights beyond fp16, at either end
        large |= mx > m + SLACK && fabsf(mx) >= LARGE;
        m = mn;
        l *= alpha;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
          for (int r = 0; r < 16; ++r) o[t][r] *= alpha;
      }
      // granule by granule: the probabilities of one beside the second product
      // of the one before
      v8h fp[GR], fv[NPV];
      float km[GR], cm[GR], sum[GR] = {};
#pragma unroll
      for (int i = 0; i < GR; ++i) {
        km[i] = kmul_of(g, i);
        cm[i] = exponent_of(g, i) - (m - (FP16_TOP - SLACK));
      }
      auto weights = [&](int i, int j) __attribute__((always_inline)) {   // scores j, j + 1 of granule i
        const v16f& x = sc[i >> 1];
        const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(x[8 * (i & 1) + j], km[i], cm[i]));
        const float z = __builtin_amdgcn_exp2f(__builtin_fmaf(x[8 * (i & 1) + j + 1], km[i], cm[i]));
        // float32, not the rounded weights: where another block's values are
        // larger by many powers of two, fp16 holds a weight's share of the
        // product, but not its share of the sum
        sum[i] += y + z;
        asm volatile("" : "+v"(sum[i]));   // here, beside the MFMAs, not behind them
        fp[i][j] = (_Float16)y;
        fp[i][j + 1] = (_Float16)z;
      };
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) fv[j] = value(j);
#pragma unroll
      for (int j = 0; j < 8; j += 2) weights(0, j);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < NPV; ++j) {
        const int i = j / DT, t = j % DT;
        o[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fv[j], fp[i], o[t], 0, 0, 0);
        if (j + AHEAD < NPV) fv[j + AHEAD] = value(j + AHEAD);
        if (i + 1 < GR)
#pragma unroll
          for (int e = 8 * t / DT; e < 8 * (t + 1) / DT; e += 2) weights(i + 1, e);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int i = 0; i < GR; ++i) l = __builtin_fmaf(sum[i], vinv_of(g, i), l);
    };

    if (turns > 0) {
      int blk1 = load_block(1), blk2;        // the next unit's blocks, and the one's after it
      Granules g0, g1;
      Codes c;
      {
        const int blk0 = load_block(0);
        g0 = load_granules(blk0);
        c = load_codes(0, blk0);
        blk2 = load_block(2);
        clear_codes(0, c, blk0);
#pragma unroll
        for (int j = 0; j < 4 * LOADS; ++j) store_codes(c, j, std::integral_constant<int, 0>{});
      }
      if (turns > 1) {
        g1 = load_granules(blk1);
        c = load_codes(1, blk1);
      }
      __syncthreads();
      auto unit = [&](int u, auto buf) __attribute__((always_inline)) {
        const Granules g = g0;
        if (u + 1 < turns) clear_codes(u + 1, c, blk1);
        g0 = g1;
        compute(u, scales_of(g), c, buf, [&]() __attribute__((always_inline)) {
          blk1 = blk2;
          if (u + 2 < turns) {
            g1 = load_granules(blk1);
            c = load_codes(u + 2, blk1);
            blk2 = load_block(u + 3);
          }
        });
        __syncthreads();   // unit u + 1 is in LDS; unit u is read by every wave
      };
      int u = 0;
      for (; u + 1 < turns; u += 2) {
        unit(u, std::integral_constant<int, 0>{});
        unit(u + 1, std::integral_constant<int, 1>{});
      }
      if (u < turns) unit(u, std::integral_constant<int, 0>{});
    }

    // A row with large scores is left to FewRows, which subtracts the maximum from scores
    // that are rounded as it was. (Rounding the scores so here, in a branch of each unit,
    // costs the mixed batch 3 %, these flags 12 prompts of 200 tokens 2 %: 13.6 -> 13.9 us.)
    bool any_large = false;
    if (turns > 0) {
      int* const flags = large_flags(lds_all);
      if (half == 0) flags[PROWS * set + 32 * wave + col] = large && m < INFINITY;   // (infinite: NaN either way)
      __syncthreads();
      int any = 0;
#pragma unroll
      for (int i = 0; i < SETS * PROWS; i += 64) any |= flags[i + lane];
      any_large = __ballot(any != 0) != 0;
      large = is_large(flags, 32 * wave + col);
    }

    if constexpr (SETS > 1) {
      static_assert(64 * PWAVES * (64 * DT + 8) <= LDS_BYTES - FLAG_BYTES, "beside the flags");
      // the sets' results, lane for lane: the second's go through LDS
      constexpr int THREADS = 64 * PWAVES;
      v4f* const to = reinterpret_cast<v4f*>(lds_all) + tid;
      float* const stats = reinterpret_cast<float*>(lds_all + 16 * THREADS * 4 * DT) + tid;
      if (set > 0) {
        stats[0] = m;
        stats[THREADS] = l;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
          for (int a = 0; a < 4; ++a) to[(4 * t + a) * THREADS] = v4f{o[t][4 * a], o[t][4 * a + 1], o[t][4 * a + 2], o[t][4 * a + 3]};
      }
      __syncthreads();
      if (set > 0) return any_large;
      const float m1 = stats[0], mn = fmaxf(m, m1), a0 = __builtin_amdgcn_exp2f(m - mn), a1 = __builtin_amdgcn_exp2f(m1 - mn);
      m = mn;
      l = l * a0 + stats[THREADS] * a1;
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const v4f x = to[(4 * t + a) * THREADS];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][4 * a + e] = o[t][4 * a + e] * a0 + x[e] * a1;
        }
    }
    l = sum_halves(l);
    if (row >= w.rows || large) return any_large;
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
        part.m[r0] = m - (FP16_TOP - SLACK);   // what o and l are relative to
        part.l[r0] = l;
      }
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int a = 0; a < 4; ++a)
          *reinterpret_cast<v4f*>(&part.o[r0][32 * t + 8 * a + 4 * half]) =
              v4f{o[t][4 * a], o[t][4 * a + 1], o[t][4 * a + 2], o[t][4 * a + 3]};
    }
    return any_large;
  }

  static __device__ __forceinline__ void run(const AttnArgs& p, int splits, uint8_t* lds_all) {
    const int head = (int)(blockIdx.x % (unsigned)p.Hk);
    const int64_t rest = blockIdx.x / (unsigned)p.Hk;
    const int z = (int)(rest % splits);
    Work w;
    if (!find_work(p, rest / splits, w)) return;

    const int64_t u_lo = w.lo / U, u_hi = w.hi > w.lo ? (w.hi + U - 1) / U : u_lo;
    if (w.rows - w.row0 <= FEW_ROWS) {
      few_rows<false>(p, splits, lds_all, w, head, z, u_lo, u_hi);
      return;
    }
    if (__builtin_expect(many_rows(p, splits, lds_all, w, head, z, u_lo, u_hi), 0)) {
      __syncthreads();   // the sets' results are read
      few_rows<true>(p, splits, lds_all, w, head, z, u_lo, u_hi);
    }
  }
};

template <int D, int SETS>
__global__ __launch_bounds__(SETS * PWAVES * 64, D == 64 && SETS == 1 ? 3 : 2)
void attention_prefill_kernel(AttnArgs p, int splits) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[Prefill<D, SETS>::LDS_BYTES];
  Prefill<D, SETS>::run(p, splits, lds);
}

// Joins the pieces of a split launch: workgroup (x, y) takes every gridDim.y-th
// row from y on of row tile and key head x
template <int D>
__global__ __launch_bounds__(JOIN_THREADS)
void attention_prefill_join_kernel(AttnArgs p, int splits) {
  __shared__ __attribute__((aligned(16))) JoinSpace<D> lds;
  const int64_t item = blockIdx.x / (unsigned)p.Hk;
  const int head = (int)(blockIdx.x % (unsigned)p.Hk);
  Work w;
  if (!find_work(p, item, w)) return;
  const PartialTile<D>* const parts = reinterpret_cast<const PartialTile<D>*>(p.workspace) + item * splits * p.Hk + head;
  const int64_t left = w.rows - w.row0;
  join_rows<D>(
      lds, blockIdx.y, gridDim.y, left < PROWS ? (int)left : PROWS, splits,
      [&](int z) __attribute__((always_inline)) -> const PartialTile<D>& { return parts[(int64_t)z * p.Hk]; },
      [&](int r, int d, float sum, v4f acc) __attribute__((always_inline)) {
        const float inv = inverse_sum(sum);
        uint16_t* const dst = p.out + row_offset(w.begin, w.row0 + r, head, p.group, D, p.ldo) + d;
        *reinterpret_cast<v2u*>(dst) = v2u{pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv)};
      });
}

template <int D>
hipError_t launch(const AttnArgs& p, hipStream_t stream) {
  const int64_t items = ((p.seq.T * p.group) >> 7) + p.seq.S, pairs = items * p.Hk;
  // Up to 128 workgroups: split, into pieces of at least four units where the rows
  // may see that many (200 rows of 8 heads over 2 after 1800 tokens: 17.4 us, with
  // eight units 21.5; with up to 1024 workgroups instead of 512, 1250 rows of 32
  // heads over 4, D 64, take 44 us instead of 35: the partial results' way
  // through memory costs more than the CUs gain). Up to 512, which leave CUs a
  // workgroup or two: two sets of waves in each (us with two sets / one / split:
  // 1000 rows of 32 heads over 4, D 128, 26.4 / - / 36.4; 1500 rows over 8 heads
  // 37 / 43 / 57; 1250 rows, D 64, 28 / 33 / 43). More: one set (4632 rows of
  // 64 heads 382, with two sets 428). From 257 on also where rows see too little to
  // be shared out (us with one / two sets, single tokens, 8 heads: 41 sequences of 39
  // tokens 5.6 / 9.1, 40 of up to 900 17.2 / 20.7; 12 prompts of 200 12.2 / 17.0; 6 of 400
  // after up to 500 21.2 / 23.7), unless FewRows has two tiles a workgroup (30
  // sequences of up to 900 tokens, 32 rows a head 26.8 / 21.4).
  const int64_t longest = reach(p) / (4 * UNIT);
  int64_t splits = pairs > 128 ? 1 : SPLIT_GROUPS / pairs;
  if (splits > longest) splits = longest;
  if (splits < 1) splits = 1;
  const int64_t rows = p.seq.T * p.group, S = p.seq.S;
  const bool share = reach(p) >= 1024 || (rows > 16 * S && rows <= FEW_ROWS * S);
  const bool two = splits == 1 && pairs <= (share ? 512 : 256);
  if (pairs * splits > 0x7FFFFFFF) return hipErrorInvalidValue;
  if (two)
    hipLaunchKernelGGL((attention_prefill_kernel<D, 2>), dim3((unsigned)(pairs * splits)), dim3(2 * PWAVES * 64), 0, stream, p, (int)splits);
  else
    hipLaunchKernelGGL((attention_prefill_kernel<D, 1>), dim3((unsigned)(pairs * splits)), dim3(PWAVES * 64), 0, stream, p, (int)splits);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  hipLaunchKernelGGL((attention_prefill_join_kernel<D>), dim3((unsigned)pairs, 16), dim3(JOIN_THREADS), 0, stream, p, (int)splits);
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
