// Internal declarations shared by the library's translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace iqp {

// Arguments of the fused indexer-Q kernel (validated on the host).
struct IndexerQArgs {
  const uint8_t* a;              // E4M3 activations [M, K], row stride lda bytes
  int64_t lda;
  const uint8_t* a_scale_bytes;  // packed UE8M0 words viewed as bytes
  int64_t as_sm, as_sw;          // word strides (int32 units)
  const uint8_t* w;              // E4M3 weights [H*128, K], row stride ldw bytes
  int64_t ldw;
  const uint8_t* w_scales;       // UE8M0 [H, K/128]
  int64_t M;
  int32_t nkb;                   // K / 128
  int32_t H;
  const int64_t* positions;      // [M]
  const float* cos_sin;          // [max_pos, 64]
  int64_t max_pos;
  const float* cos_sin_lanes;    // null, or the table's lane-ordered copy (launch_rope_table_lanes),
                                 // which the split-role kernel then reads instead of cos_sin
  uint8_t* q_fp4;                // [M, H, 64]
  uint8_t* q_scales;             // [M, H, 4]
  float* dbg;                    // [M, H*128] for the diagnostic stages
  const uint16_t* x;             // bf16 activations [M, K], row stride ldx elements (one-launch small path)
  int64_t ldx;
  int32_t chunks;                // token chunks per head pair (set by the launcher)
  // one-launch kernel: the packed FP8 quantization of an independent bf16
  // matrix [side_words / side_nw rows, K] run by extra workgroups of the
  // same launch (none when side_words == 0); layout and strides as in
  // launch_fp8_quant
  const uint16_t* side_x;
  int64_t side_ldx;
  uint8_t* side_q;
  int64_t side_ldq;
  int32_t* side_scales;
  int64_t side_sm, side_sw;
  int32_t side_nw, side_nkb;
  int64_t side_words;
  // small-batch kernel, split over K (null: not split): the workspace, of
  // splitk_ws_bytes >= splitk_workspace_bytes(H) bytes, zero before its first
  // use and left zero by every call (the counters); calls sharing one must
  // not overlap
  uint8_t* splitk_ws;
  int64_t splitk_ws_bytes;
};

// the one-launch kernel's split-K workspace: the counters (one per head and
// 32-token tile), then each split's float32 partial sums of every head and
// tile (at most 4 sets of 16 KiB a head: 3 splits x 1 tile, 2 x 2). The
// counter region is sized by the workspace, for the most heads it can hold
// (8 bytes a head, in 256-byte units), so that calls with different head
// counts find their counters in one region and may share a workspace.
constexpr int64_t SPLITK_MIN_TOKENS = 12;
constexpr int64_t SPLITK_MAX_TOKENS = 64;
__host__ __device__ constexpr int64_t splitk_counter_bytes(int64_t H) { return (8 * H + 255) / 256 * 256; }
__host__ __device__ constexpr int64_t splitk_workspace_bytes(int64_t H) { return splitk_counter_bytes(H) + 65536 * H; }
__host__ __device__ constexpr int64_t splitk_counter_region(int64_t ws_bytes) {
  return splitk_counter_bytes(ws_bytes / (65536 + 8));
}

hipError_t launch_fp8_quant(const uint16_t* x, int64_t M, int64_t K, int64_t ldx,
                            uint8_t* q, int64_t ldq, int32_t* scales,
                            int64_t s_stride_m, int64_t s_stride_w, hipStream_t stream);

// stage -1: FP4 output; 0, 1, 2: float32 diagnostics (see iqprep.h)
hipError_t launch_indexer_q(const IndexerQArgs& args, int stage, hipStream_t stream);
// the float32 GEMM sums of the kernel that launch_indexer_q(args, -1) runs
// (its diagnostic build; the general kernel's stage 0 where that one runs)
hipError_t launch_indexer_q_gemm_dump(const IndexerQArgs& args, hipStream_t stream);
// launch_indexer_q(args, -1) with shader-clock stamps (args.dbg, uint64
// [4 * workgroups]) where it runs the split-role kernel; *workgroups is set
// first; hipErrorNotSupported where another kernel would run, and
// hipErrorInvalidValue when stamp_capacity < 4 * workgroups (nothing launched)
hipError_t launch_indexer_q_clock(const IndexerQArgs& args, int64_t stamp_capacity, int64_t* workgroups,
                                  hipStream_t stream);
// FP4 output with convention variant v (bit 0: interleaved RoPE pairs, bit 1:
// OCP floor-rule FP4 scales, bit 2: per-row weight scales); v = 0 is
// launch_indexer_q(args, -1, stream); otherwise the variant build of the
// small-batch or pipelined kernel where the default call would run that
// kernel (per-row weight scales in the pipelined one: 4-byte aligned), and
// the general kernel everywhere else
hipError_t launch_indexer_q_variant(const IndexerQArgs& args, int variant, hipStream_t stream);

// the pipelined FP4-output kernel (indexer_q_pipe.hip) for the shapes it takes
// (K = 1536, token counts that fit in 31 bits); args.chunks set
bool indexer_q_pipe_supported(const IndexerQArgs& args);
hipError_t launch_indexer_q_pipe(const IndexerQArgs& args, hipStream_t stream);
// the same kernel with convention variant v = 1..7 compiled in
// (indexer_q_pipe_v<v>.hip; bits as in launch_indexer_q_variant; v >= 4 needs
// 4-byte aligned weight scales)
hipError_t launch_indexer_q_pipe_v1(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_pipe_v2(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_pipe_v3(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_pipe_v4(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_pipe_v5(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_pipe_v6(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_pipe_v7(const IndexerQArgs& args, hipStream_t stream);

// the split-role build of the pipelined kernel (indexer_q_split.hip): the
// pipelined kernel's shapes and arguments, table positions below 2^31
bool indexer_q_split_supported(const IndexerQArgs& args);
hipError_t launch_indexer_q_split(const IndexerQArgs& args, hipStream_t stream);
// the same kernel reading the RoPE rows from args.cos_sin_lanes (indexer_q_split_lanes.hip)
hipError_t launch_indexer_q_split_lanes(const IndexerQArgs& args, hipStream_t stream);
// the split-role kernel with convention variant v = 1..3 compiled in
// (indexer_q_split_v<v>.hip; per-row weight scales do not fit its registers);
// where indexer_q_split_supported holds
hipError_t launch_indexer_q_split_v1(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_split_v2(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_split_v3(const IndexerQArgs& args, hipStream_t stream);

// diagnostic builds: the float32 GEMM sums (Q before RoPE) of the pipelined,
// split-role and small-batch kernels' K loops in args.dbg [M, H*128]; the
// pipelined and split ones take the arguments of their FP4 launchers
// (args.chunks set); the small-batch one quantizes bf16 args.x itself when
// that is set (the one-launch kernel), else reads args.a
hipError_t launch_indexer_q_pipe_dump(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_split_dump(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_small_dump(const IndexerQArgs& args, hipStream_t stream);
// the split-role FP4 kernel with four uint64 stamps per workgroup in args.dbg
// (s_memtime start, end; s_memrealtime start, end; zeros for a workgroup with
// no tiles); args.chunks set
hipError_t launch_indexer_q_split_clock(const IndexerQArgs& args, hipStream_t stream);
// the same stamps from the build reading args.cos_sin_lanes (indexer_q_split_lanes_clock.hip)
hipError_t launch_indexer_q_split_lanes_clock(const IndexerQArgs& args, hipStream_t stream);

// the small-batch FP4-output kernel (indexer_q_small.hip): K = 1536, 1 to 256
// tokens, weight scales 4-byte aligned
bool indexer_q_small_supported(const IndexerQArgs& args);
hipError_t launch_indexer_q_small(const IndexerQArgs& args, hipStream_t stream);
// the same kernel with convention variant v = 1..7 compiled in
// (indexer_q_small_v<v>.hip; bits as in launch_indexer_q_variant)
hipError_t launch_indexer_q_small_v1(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_small_v2(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_small_v3(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_small_v4(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_small_v5(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_small_v6(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_small_v7(const IndexerQArgs& args, hipStream_t stream);
// the same kernel quantizing bf16 activations (args.x, args.ldx) itself: one
// launch from X to FP4 Q; K = 1536, 1 to 256 tokens
// (with args.splitk_ws set and SPLITK_MIN_TOKENS to SPLITK_MAX_TOKENS
// tokens, its split-K build)
bool indexer_q_small_bf16_supported(const IndexerQArgs& args);
hipError_t launch_indexer_q_small_bf16(const IndexerQArgs& args, hipStream_t stream);
// the same with convention variant v = 1..7 compiled in (indexer_q_small_v<v>.hip),
// and a dispatcher over v = 0..7 (0: launch_indexer_q_small_bf16)
hipError_t launch_indexer_q_small_bf16_v1(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_small_bf16_v2(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_small_bf16_v3(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_small_bf16_v4(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_small_bf16_v5(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_small_bf16_v6(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_small_bf16_v7(const IndexerQArgs& args, hipStream_t stream);
hipError_t launch_indexer_q_small_bf16_variant(const IndexerQArgs& args, int variant, hipStream_t stream);

// standalone epilogue: bf16 Q [M, H*128] (row stride ldq elements) -> RoPE,
// Hadamard-128, FP4 codes [M, H, 64] and scale bytes [M, H, 4]
// (interleaved: RoPE pairs (2i, 2i+1); floor_rule: OCP MX FP4 scales)
hipError_t launch_indexer_q_epilogue(const uint16_t* q, int64_t ldq, int64_t M, int32_t H,
                                     const int64_t* positions, const float* cos_sin, int64_t max_pos,
                                     uint8_t* q_fp4, uint8_t* q_scales, bool interleaved, bool floor_rule,
                                     hipStream_t stream);

// weight preparation: bf16 [N, K] -> E4M3 [N, K] + UE8M0 [N/128, K/128]
hipError_t launch_fp8_quant_weight(const uint16_t* w, int64_t N, int64_t K, int64_t ldw, uint8_t* q, int64_t ldq,
                                   uint8_t* scales, int64_t ld_scales, hipStream_t stream);

// --- the operators around an attention layer ---------------------------------

// A ragged batch over the paged cache: sequence s has the rows cu[s] ..
// cu[s + 1] - 1 of the batch's T rows, which are its last tokens: the last of
// them is at position lens[s] - 1. Its token at position p lives at
// p % 2^log_block of block table[s * ld_table + p / 2^log_block] (an entry
// outside [0, n_blocks): not held).
struct SeqBatch {
  const int32_t* cu;        // [S + 1]
  const int32_t* lens;      // [S]
  const int32_t* table;     // [S, max_blocks], row stride ld_table
  int64_t ld_table;
  int64_t T;
  int64_t n_blocks;
  int32_t S;
  int32_t max_blocks;
  int32_t log_block;
};

// Arguments of the block-scaled FP8 product (validated on the host).
struct Fp8GemmArgs {
  const uint8_t* a;         // E4M3 [M, K], row stride lda bytes
  int64_t lda;
  const int32_t* a_scales;  // packed UE8M0 words, strides in words
  int64_t as_sm, as_sw;
  const uint8_t* w;         // E4M3 [N, K], row stride ldw bytes
  int64_t ldw;
  const uint8_t* w_scales;  // UE8M0 [ceil(N / 128), K / 128], row stride ld_ws
  int64_t ld_ws;
  int64_t M, N;
  int32_t nkb;              // K / 128
  uint16_t* out;            // bf16 [M, N], row stride ldo elements
  int64_t ldo;
  bool wide_out;            // 16-byte stores allowed (out and ldo aligned)
  int32_t splits;           // pieces of the K blocks: fp8_gemm_splits(M, N, K), or 1 without a workspace
  float* sums;              // workspace of a split product
};
// workgroups of a split product at most, each with a 64x64 tile of float32 sums
constexpr int GEMM_SPLIT_GROUPS = 256;
constexpr int64_t GEMM_WORKSPACE_BYTES = (int64_t)GEMM_SPLIT_GROUPS * 64 * 64 * 4;
int fp8_gemm_splits(int64_t M, int64_t N, int64_t K);
// The product's kernels: weight rows x tokens of a workgroup.
enum GemmKernel {
  GEMM_STREAM_16x16,
  GEMM_STREAM_32x16,
  GEMM_STREAM_16x32,
  GEMM_STREAM_32x32,
  GEMM_STREAM_16x64,
  GEMM_STREAM_32x64,
  GEMM_SPLIT_64x64,
  GEMM_TILE_64x64,
  GEMM_TILE_128x64,
  GEMM_TILE_128x128,        // four LDS stages
  GEMM_TILE_128x128_TWO,    // two, so that two workgroups share a CU
  GEMM_TILE_256x256,
};
// the one that a product takes, in `splits` pieces of its K blocks
GemmKernel fp8_gemm_kernel(int64_t M, int64_t N, int64_t K, int splits);
const char* fp8_gemm_kernel_name(GemmKernel kernel);
hipError_t launch_fp8_gemm(const Fp8GemmArgs& args, hipStream_t stream);

struct QkNormRopeArgs {
  const uint16_t* q;        // bf16 [M, Hq * D], row stride ldq
  const uint16_t* k;        // bf16 [M, Hk * D], row stride ldk
  int64_t ldq, ldk;
  const uint16_t* q_weight; // bf16 [D]
  const uint16_t* k_weight;
  const int64_t* positions; // [M]
  const float* cos_sin;     // [max_pos, rope_dim]
  int64_t max_pos;
  uint16_t* q_out;
  uint16_t* k_out;
  int64_t ldqo, ldko;
  int64_t M;
  int32_t Hq, Hk, rope_dim;
  float eps;
};
// D: 64, 128 or 256
hipError_t launch_qk_norm_rope(const QkNormRopeArgs& args, int D, bool interleaved, hipStream_t stream);

struct KvAppendArgs {
  SeqBatch seq;
  const uint16_t* k;        // bf16 [T, Hk * D], row stride ldk
  const uint16_t* v;
  int64_t ldk, ldv;
  uint8_t* k_cache;         // E4M3 [n_blocks, Hk, B, D]
  uint8_t* v_cache;         // E4M3 [n_blocks, Hk, D, B]
  uint8_t* k_scales;        // UE8M0 [n_blocks, Hk]
  uint8_t* v_scales;
  int32_t Hk;
};
// D: 64 or 128
hipError_t launch_kv_append(const KvAppendArgs& args, int D, hipStream_t stream);

struct KvReadArgs {
  SeqBatch seq;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  uint16_t* k_out;          // bf16 [T, Hk * D], row stride ldk
  uint16_t* v_out;
  int64_t ldk, ldv;
  int32_t Hk;
};
hipError_t launch_kv_read(const KvReadArgs& args, int D, hipStream_t stream);

// Arguments of attention over the FP8 cache (validated on the host).
struct AttnArgs {
  SeqBatch seq;
  const uint16_t* q;        // bf16 [T, Hk * group * D], row stride ldq
  int64_t ldq;
  uint16_t* out;            // bf16, laid out alike, row stride ldo
  int64_t ldo;
  const uint8_t* k_cache;   // as in KvReadArgs
  const uint8_t* v_cache;
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  int32_t Hk, group;        // key heads, query heads per key head
  int32_t window;           // 0: none
  float scale_log2;         // softmax scale * log2(e)
  uint8_t* workspace;       // attention_workspace_bytes(D)
  int64_t max_rows;         // set by the launcher: sequences of more rows (tokens * group) are the
                            // prompt kernel's, the others the decode kernel's
};
// workgroups of the decode kernel: two for each of a full chip's 256 CUs (64
// sequences of up to 8192 tokens: 112 us; with 256 workgroups 126, 768 123, 1024 116)
constexpr int ATTN_WORKGROUPS = 512;
// A batch of no more rows (tokens times query heads of a key head) than this on
// average is the decode kernel's, but see below (32 sequences of 6000 tokens, 64 heads over 8, us,
// decode / prompt kernel: 64 rows 185 / 207, 128 rows 326 / 207). Of another one,
// sequences of more rows are the prompt kernel's. These sides are of sequences alike:
// the host knows the average alone, so that a prompt's chunk beside many single tokens
// over long tables may be the decode kernel's too, which reads the cache for every 16
// rows of it (64 heads over 8, us together / single tokens alone / chunk alone: 448 new
// tokens beside 63 single ones, 8192 held, 678 / 207 / 167; 512 beside 128, 887 / 400 /
// 166; 1000 beside 64, where the average is above and both kernels run, 534 / 205 / 331).
constexpr int ATTN_DECODE_ROWS = 64;
// Where a row sees no more tokens than this, batches of few rows are the prompt
// kernel's too: a workgroup a sequence and head, no second launch (single tokens, us,
// direct / decode kernel: 10 sequences of 35 tokens 5.8 / 8.5, 30 of up to 900, 64
// heads over 8, 12.8 / 18.2, of up to 2000 20.8 / 25.3; 64 of up to 4000 84 / 69, as
// the lengths differ; 8 sequences of 2000 with 64 rows a head 28 / 25); twice as many
// tokens where ATTN_MANY_PAIRS sequences times heads even out by themselves or
// ATTN_MANY sequences make the decode kernel's walk over all lengths long (100 to 4000
// tokens: 128 sequences, 8 heads 120 / 128, 200 176 / 196; 500, one head of 64, 37 / 49,
// 1000 57 / 92; but of 2000 to 8000, 128 sequences, 8 heads, 273 / 254).
constexpr int ATTN_DIRECT_REACH = 2048, ATTN_DIRECT_ROWS = 32, ATTN_MANY_PAIRS = 1024, ATTN_MANY = 256;
// The sequences of few rows in such a batch: where a row sees no more tokens than
// this (the table, or the window), the prompt kernel takes them too, beside the
// others; else they are the decode kernel's, behind it (two prompts of 500 tokens
// beside single tokens, us, one / two kernels: 32 sequences of 2000 39 / 57, of 4000
// 71 / 81, of 7500 138 / 133; 8 of 16000 166 / 83; 24 sequences of 1 to 30 new tokens
// after up to 3900: 69 / 95).
constexpr int ATTN_SHORT_REACH = 8192;
int64_t attention_decode_workspace_bytes(int D);
int64_t attention_prefill_workspace_bytes(int D);
hipError_t launch_attention_decode(const AttnArgs& args, int D, hipStream_t stream);
hipError_t launch_attention_prefill(const AttnArgs& args, int D, hipStream_t stream);
// both kernels' workspace is the same memory: their launches follow one another
int64_t attention_workspace_bytes(int D);
hipError_t launch_attention(const AttnArgs& args, int D, hipStream_t stream);

// compute units of the current device (cached per device)
int cu_count();

hipError_t launch_rope_table(double theta, int64_t max_pos, int32_t rope_dim,
                             float* cos_sin, hipStream_t stream);
// the lane-ordered copy of a [max_pos, 64] table: ceil(max_pos / 32) * 2048 floats
// (layout in rope_table.hip)
hipError_t launch_rope_table_lanes(const float* cos_sin, int64_t max_pos, float* out, hipStream_t stream);

}  // namespace iqp
