/*
 * iqprep.h — C ABI of libiqprep.so: DeepSeek-V4 indexer-Q preparation on
 * AMD Instinct MI355X (gfx950).
 *
 * The library computes, on the GPU, the calls of indexer-Q preparation:
 *
 *   1. fp8_quant_1x128_ue8m0     packed-UE8M0 FP8 1x128 activation quantization
 *      (tokenspeed PR "perf(deepseek-v4): accelerate indexer Q and packed FP8
 *      quantization", Summary; input contract in Risk and fallback).
 *   2. indexer_q_gemm_rope_fp4   block-scaled FP8 Q projection whose epilogue
 *      applies RoPE, a 128-point Hadamard rotation and FP4 e2m1 quantization
 *      (TensorRT-LLM PR "Fuse DeepSeek-V4 Indexer Q projection with CuTe DSL",
 *      sequence diagram: FP8 input + UE8M0 scales in, packed FP4 Q and scales
 *      out; the same tokenspeed PR, Summary: RoPE, Hadamard and FP4 make up
 *      the Q preparation); indexer_q_gemm_rope_fp4_ex takes convention flags.
 *   3. indexer_q_rope_hadamard_fp4   the same RoPE / Hadamard / FP4 epilogue as
 *      a standalone launch over a bf16 Q (the unfused chain's second half).
 *   4. indexer_q_prep_bf16   calls 1 and 2 as one launch for decode-sized
 *      batches (up to 256 tokens); indexer_q_prep_bf16_ex takes the flags;
 *      indexer_q_prep_bf16_with_quant also runs call 1 on an independent
 *      matrix in the same launch; indexer_q_prep_bf16_with_quant_ws is that
 *      call with a caller-owned workspace, which lets it split each head's
 *      K range over several workgroups at 12 to 64 tokens, and
 *      indexer_q_prep_bf16_with_quant_noalloc the same with the library's own
 *      scratch, for callers that cannot allocate.
 *   5. fp8_quant_weight_128x128_ue8m0   the weights' E4M3 codes and per-tile
 *      scales that calls 2 and 4 take (weight preparation, off the
 *      per-token path).
 *   6. iqp_rope_table_lanes   a RoPE table rearranged for the prefill kernel's
 *      16-byte loads (built once per table); indexer_q_gemm_rope_fp4_lanes
 *      is call 2 reading it.
 *
 * and the operators of the attention layer around it, with 8-bit operands:
 *
 *   7. fp8_gemm_1x128_128x128   the layer's other projections: the operands of
 *      calls 1 and 5, bf16 out.
 *   8. qk_norm_rope   RMS norm of every query and key head and RoPE, in one pass.
 *   9. kv_cache_append_fp8, kv_cache_read_fp8   a paged key/value cache in E4M3
 *      with a UE8M0 scale per block of tokens and head: written, read back.
 *  10. attention_fp8_kv   causal attention over that cache, for prompts, their
 *      continuations and single tokens in one ragged batch.
 *
 * and the products beside it whose weights depend on the token:
 *
 *  11. moe_route   the experts of every token and their weights, from the router's
 *      logits.
 *  12. group_rows   a batch's entries sorted by expert or adapter: the order that
 *      calls 13 to 16 read.
 *  13. fp8_grouped_swiglu_1x128   the experts' first product, silu(gate) * up, and
 *      the 1x128 quantization of the result.
 *  14. fp8_grouped_gemm_1x128_128x128   call 7 with weights of its own for every
 *      group of rows (the experts' second product).
 *  15. moe_combine   every token's weighted sum of its experts' rows.
 *  16. lora_add   low-rank adapters of many requests, added to a projection's output.
 *
 * Conventions shared by every entry point:
 *
 *   - Every data pointer is a caller-owned DEVICE pointer on the current HIP
 *     device. The library never allocates, frees, copies or synchronizes; it
 *     enqueues kernels on `stream` (a hipStream_t; NULL = the null stream) and
 *     returns. Calls are therefore safe to capture into a HIP graph.
 *   - Inputs are never modified (in-place outputs are: a cache, lora_add's out).
 *   - Sizes and leading dimensions are in elements of the named type unless
 *     stated otherwise; all offsets are computed in 64-bit.
 *   - Return value: IQP_OK, or an IQP_ERR_* code. Argument checks happen on
 *     the host before anything is enqueued; on any error nothing is enqueued
 *     (IQP_ERR_HIP: the launch itself failed). IQP_ERR_UNSUPPORTED means the
 *     arguments are well formed but outside the fast path's contract, and the
 *     caller should use another implementation: the library never falls back
 *     silently.
 *   - M == 0 is a successful no-op.
 *   - Entry points are reentrant and thread-safe; the only global state is a
 *     per-device cache of the device architecture, filled on first use, and
 *     the per-device scratch of indexer_q_prep_bf16_with_quant_noalloc (whose
 *     calls must not overlap on one GPU).
 *
 * Number formats: E4M3 is the OCP OFP8 "fn" variant (bias 7, max 448, no
 * infinities); E2M1 is OCP MX FP4 (magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6);
 * a UE8M0 byte b means 2^(b-127).
 */
#ifndef IQPREP_H
#define IQPREP_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define IQP_OK              0
#define IQP_ERR_INVALID     1  /* null pointer, negative size, leading dimension smaller than a row, overlapping scale strides */
#define IQP_ERR_UNSUPPORTED 2  /* well formed but outside the contract (K % 128, alignment, head shape, device): use another path */
#define IQP_ERR_HIP         3  /* a HIP runtime call or kernel launch failed */

#define IQP_ABI_VERSION     3

/* Convention flags of indexer_q_gemm_rope_fp4_ex, indexer_q_prep_bf16_ex and
 * indexer_q_rope_hadamard_fp4 (0: the defaults of indexer_q_gemm_rope_fp4).
 * The pages leave these conventions open. */
#define IQP_ROPE_INTERLEAVED     0x1  /* RoPE pairs (2i, 2i+1), i < rope_dim/2, instead of (i, i + rope_dim/2) */
#define IQP_FP4_SCALE_OCP_FLOOR  0x2  /* FP4 scale e = floor(log2 max(amax, 1e-4)) - 2 (OCP MX rule), codes
                                         saturating at +-6, instead of e = ceil(log2(amax / 6)) */
#define IQP_W_SCALES_PER_ROW     0x4  /* the projection calls only (not the standalone epilogue): w_scales holds one UE8M0 byte per
                                         weight row and K block, [H*D, K/128] row-major, instead of one per
                                         128x128 tile */

/*
 * fp8_quant_1x128_ue8m0 — packed-UE8M0 FP8 activation quantization.
 *
 * tokenspeed PR "perf(deepseek-v4): accelerate indexer Q and packed FP8
 * quantization", Summary (an online FP8 quantizer for DeepGEMM activations
 * with UE8M0 scale exponents packed into int32 words) and Risk and fallback
 * (a contiguous, aligned BF16 matrix with K divisible by 128; the existing
 * tiny-scale floor is kept).
 *
 * For every row m and 128-element block j of x:
 *   amax = max(max_k |x[m, 128j+k]|, 1e-4)          (1e-4: the tiny-scale floor)
 *   e    = ceil(log2(amax / 448))                     exact; -22 <= e <= 120
 *   q[m, 128j+k] = E4M3 round-to-nearest-even of x * 2^-e   (never saturates)
 *   byte(m, j) = e + 127
 * Four consecutive block bytes form one int32 word, block 4w+t in byte t
 * (little-endian): word (m, w) = scales[m * s_stride_m + w * s_stride_w], for
 * 0 <= w < ceil(K/512). Bytes for blocks past K/128 are written as zero.
 *
 *   x        bf16 [M, K], row stride ldx (elements, >= K); 16-byte aligned and
 *            ldx a multiple of 8, else IQP_ERR_UNSUPPORTED.
 *   q        E4M3 bytes [M, K], row stride ldq (bytes, >= K); 8-byte aligned
 *            and ldq a multiple of 8, else IQP_ERR_UNSUPPORTED.
 *   scales   int32 words, 4-byte aligned. Strides in int32 units; the two
 *            supported layouts are K-major (s_stride_w == 1, s_stride_m >=
 *            ceil(K/512)) and MN-major (s_stride_m == 1, s_stride_w >= M);
 *            anything else is IQP_ERR_INVALID.
 *   K        multiple of 128, else IQP_ERR_UNSUPPORTED.
 *
 * Inputs must be finite (NaN / Inf are outside the contract).
 */
int fp8_quant_1x128_ue8m0(const void* x, int64_t M, int64_t K, int64_t ldx,
                          void* q, int64_t ldq,
                          int32_t* scales, int64_t s_stride_m, int64_t s_stride_w,
                          void* stream);

/*
 * indexer_q_gemm_rope_fp4 — fused block-scaled FP8 Q projection + RoPE +
 * Hadamard-128 + FP4 e2m1 quantization, one launch.
 *
 * TensorRT-LLM PR "Fuse DeepSeek-V4 Indexer Q projection with CuTe DSL",
 * sequence diagram (FP8 input and UE8M0 scales from the quantizer feed a GEMM
 * with a RoPE and FP4 epilogue that returns packed FP4 Q and scales) and
 * Description / Paths compared (the unfused chain: Q GEMM, RoPE kernel, FP4
 * quantization kernel, scale copies); tokenspeed PR "perf(deepseek-v4):
 * accelerate indexer Q and packed FP8 quantization", Summary (the Hadamard
 * transform belongs to the optimized Q preparation).
 *
 * For every token m and head h (n = 128h + d, 0 <= d < 128):
 *   Q[m, n]  = sum_j 2^(ea(m,j) + ew(h,j)) * sum_{k in block j} A[m,k] W[n,k]
 *              (float32 accumulation)
 *   RoPE     for i < 32, p = positions[m], c = cos_sin[p, i], s = cos_sin[p, 32+i]:
 *              y_i = Q_i c - Q_{i+32} s,  y_{i+32} = Q_{i+32} c + Q_i s;  y_d = Q_d for d >= 64
 *   Hadamard z = (H_128 / sqrt(128)) y,  H[r][c] = (-1)^popcount(r & c)
 *   FP4      per 32-element block b: amax = max(max |z|, 1e-4),
 *              e = ceil(log2(amax / 6)) (so e >= -15), q_scales[m, h, b] = e + 127,
 *              codes = E2M1 round-to-nearest-even of z * 2^-e; two codes per
 *              byte, element 2t in the low nibble.
 * Q is never written to memory in any precision.
 *
 *   a          E4M3 [M, K] from fp8_quant_1x128_ue8m0, row stride lda (bytes);
 *              16-byte aligned, lda a multiple of 16.
 *   a_scales   the packed scale words that call wrote, with its strides
 *              (as_stride_m, as_stride_w), same layout rules.
 *   w          E4M3 weights [H*D, K], K contiguous, row stride ldw (bytes);
 *              16-byte aligned, ldw a multiple of 16.
 *   w_scales   UE8M0 bytes [H*D/128, K/128], row-major (one per 128x128 tile).
 *   M          tokens (>= 0); K: multiple of 128, at most 32768; H >= 1; D must
 *              be 128 and rope_dim 64 (else IQP_ERR_UNSUPPORTED). Row strides
 *              below 2^23 bytes and scale-word strides with
 *              as_stride_m < 2^20, (K/512) * as_stride_w < 2^28 (else
 *              IQP_ERR_UNSUPPORTED).
 *   positions  int64 [M]. A position outside [0, max_pos) is a precondition
 *              violation: it is clamped into range (the row's output is then
 *              meaningless, but no memory outside the table is read).
 *   cos_sin    float32 [max_pos, rope_dim]: cos of the rotation angles in
 *              columns [0, rope_dim/2), sin in [rope_dim/2, rope_dim); any
 *              frequencies may be used (iqp_rope_cos_sin_table builds the
 *              standard ones). 16-byte aligned; max_pos >= 1.
 *   q_fp4      uint8 [M, H, D/2] packed E2M1 codes, 16-byte aligned.
 *   q_scales   uint8 [M, H, D/32] UE8M0 bytes, 4-byte aligned.
 *
 * Q must fit float32: the output is undefined if |Q| would overflow, which
 * needs an exponent sum ea + ew near 99 or above (|A W| <= 448^2 per term);
 * activations from fp8_quant_1x128_ue8m0 and weights of ordinary magnitude
 * are far inside that range.
 */
int indexer_q_gemm_rope_fp4(const void* a, int64_t lda,
                            const int32_t* a_scales, int64_t as_stride_m, int64_t as_stride_w,
                            const void* w, int64_t ldw,
                            const uint8_t* w_scales,
                            int64_t M, int64_t K, int32_t H, int32_t D, int32_t rope_dim,
                            const int64_t* positions,
                            const float* cos_sin, int64_t max_pos,
                            uint8_t* q_fp4, uint8_t* q_scales,
                            void* stream);

/*
 * indexer_q_gemm_rope_fp4_ex — indexer_q_gemm_rope_fp4 with convention flags.
 *
 * The same pages as indexer_q_gemm_rope_fp4: they name the MLA RoPE kernel
 * and MX-style FP4 block scales but fix neither the RoPE pair layout nor the
 * scale rule. flags 0 is exactly indexer_q_gemm_rope_fp4 (same kernels, same
 * output). Otherwise, with the arguments, layouts and errors of that call:
 *   IQP_ROPE_INTERLEAVED      pair i < 32 is (Q_2i, Q_2i+1), rotated by the
 *                             angle of table columns i and 32 + i as before;
 *   IQP_FP4_SCALE_OCP_FLOOR   e = floor(log2 max(amax, 1e-4)) - 2 (so e >= -16),
 *                             codes = E2M1 RNE of z * 2^-e saturated at +-6;
 *   IQP_W_SCALES_PER_ROW      w_scales is UE8M0 [H*D, K/128] row-major (one
 *                             byte per weight row n and K block j), and the
 *                             projection uses ew(n, j) in place of ew(h, j).
 * Other bits: IQP_ERR_INVALID. Where the base call would run one of the
 * K = 1536 production kernels (small-batch up to 256 tokens, pipelined
 * above) the flags run that kernel's variant build (per-row weight scales
 * in the pipelined one need w_scales 4-byte aligned; flags without
 * IQP_W_SCALES_PER_ROW run its split-role build, with it the one-role one);
 * otherwise the general tiled kernel runs (slower than the
 * K = 1536 production kernels).
 */
int indexer_q_gemm_rope_fp4_ex(const void* a, int64_t lda,
                               const int32_t* a_scales, int64_t as_stride_m, int64_t as_stride_w,
                               const void* w, int64_t ldw,
                               const uint8_t* w_scales,
                               int64_t M, int64_t K, int32_t H, int32_t D, int32_t rope_dim,
                               const int64_t* positions,
                               const float* cos_sin, int64_t max_pos,
                               uint8_t* q_fp4, uint8_t* q_scales,
                               int32_t flags, void* stream);

/*
 * indexer_q_gemm_rope_fp4_lanes — indexer_q_gemm_rope_fp4 (default
 * conventions) that takes, beside the table, its lane-ordered copy from
 * iqp_rope_table_lanes (built once per table, like the weights).
 *
 * The same pages and the same computation: RoPE on the indexer Q with a
 * cos/sin table (tokenspeed PR "perf(deepseek-v4): accelerate indexer Q and
 * packed FP8 quantization", Summary; TensorRT-LLM PR "Fuse DeepSeek-V4
 * Indexer Q projection with CuTe DSL", sequence diagram). The output is
 * byte for byte that of indexer_q_gemm_rope_fp4 with the same arguments:
 * where that call runs the split-role K = 1536 kernel (257 tokens and
 * more) the rows are read from cos_sin_lanes, elsewhere from cos_sin. The
 * copy pays where a 32-token sub-tile's positions run consecutively (prefill;
 * 16-byte loads then read whole 1 KiB segments instead of gathering 32 rows);
 * for scattered positions it is somewhat slower than the table itself.
 *
 *   cos_sin_lanes  float32, ceil(max_pos / 32) * 2048 elements, 16-byte
 *                  aligned, filled by iqp_rope_table_lanes from this cos_sin
 *                  and max_pos (any other content gives undefined output);
 *                  NULL: IQP_ERR_INVALID.
 * Every other argument, layout and error is that of indexer_q_gemm_rope_fp4.
 */
int indexer_q_gemm_rope_fp4_lanes(const void* a, int64_t lda,
                                  const int32_t* a_scales, int64_t as_stride_m, int64_t as_stride_w,
                                  const void* w, int64_t ldw,
                                  const uint8_t* w_scales,
                                  int64_t M, int64_t K, int32_t H, int32_t D, int32_t rope_dim,
                                  const int64_t* positions,
                                  const float* cos_sin, const float* cos_sin_lanes, int64_t max_pos,
                                  uint8_t* q_fp4, uint8_t* q_scales,
                                  void* stream);

/*
 * indexer_q_prep_bf16 — the whole indexer-Q preparation in one launch for
 * decode-sized batches: bf16 activations in, packed FP4 Q and scales out.
 *
 * tokenspeed PR "perf(deepseek-v4): accelerate indexer Q and packed FP8
 * quantization", Summary and Perf (small shapes are kept off the multi-launch
 * path); TensorRT-LLM PR "Fuse DeepSeek-V4 Indexer Q projection with CuTe
 * DSL", kernel routing (a dedicated small-M route) and sequence diagram (FP8
 * quantization of the input, then the GEMM with the RoPE / FP4 epilogue).
 *
 * Computes exactly fp8_quant_1x128_ue8m0 on x followed by
 * indexer_q_gemm_rope_fp4 on its result (the same codes, scales and
 * rounding), without writing the FP8 activations anywhere.
 *
 *   x          bf16 [M, K], row stride ldx (elements, >= K); 16-byte aligned
 *              and ldx a multiple of 8.
 *   w, ldw, w_scales, H, D, rope_dim, positions, cos_sin, max_pos, q_fp4,
 *   q_scales   as in indexer_q_gemm_rope_fp4 (w_scales 4-byte aligned here).
 *   M          0 (no-op) to 256 tokens; K must be 1536; ldw below 2^22 bytes;
 *              H <= 65535. Anything else is IQP_ERR_UNSUPPORTED: a caller
 *              with more tokens uses the two calls above.
 */
int indexer_q_prep_bf16(const void* x, int64_t ldx, const void* w, int64_t ldw,
                        const uint8_t* w_scales,
                        int64_t M, int64_t K, int32_t H, int32_t D, int32_t rope_dim,
                        const int64_t* positions, const float* cos_sin, int64_t max_pos,
                        uint8_t* q_fp4, uint8_t* q_scales, void* stream);

/*
 * indexer_q_prep_bf16_ex — indexer_q_prep_bf16 with the convention flags of
 * indexer_q_gemm_rope_fp4_ex (same pages, same meaning: IQP_ROPE_INTERLEAVED,
 * IQP_FP4_SCALE_OCP_FLOOR, IQP_W_SCALES_PER_ROW with w_scales [H*D, K/128]
 * row-major, 4-byte aligned). flags 0 is exactly indexer_q_prep_bf16; the
 * output equals fp8_quant_1x128_ue8m0 followed by indexer_q_gemm_rope_fp4_ex
 * with the same flags. Other bits: IQP_ERR_INVALID; the other arguments,
 * limits and errors are those of indexer_q_prep_bf16.
 */
int indexer_q_prep_bf16_ex(const void* x, int64_t ldx, const void* w, int64_t ldw,
                           const uint8_t* w_scales,
                           int64_t M, int64_t K, int32_t H, int32_t D, int32_t rope_dim,
                           const int64_t* positions, const float* cos_sin, int64_t max_pos,
                           uint8_t* q_fp4, uint8_t* q_scales, int32_t flags, void* stream);

/*
 * indexer_q_prep_bf16_with_quant — indexer_q_prep_bf16 (default conventions)
 * and fp8_quant_1x128_ue8m0 of an independent bf16 matrix x2 in ONE launch:
 * extra workgroups of the one-launch kernel quantize x2 (a decode step's
 * other activation, e.g. the [M, 7168] input of a wider projection) while
 * the others prepare Q, saving a launch per step (tokenspeed PR
 * "perf(deepseek-v4): accelerate indexer Q and packed FP8 quantization",
 * Performance: the packed quantizer and the Q preparation timed as a decode
 * CUDA Graph replay per step; Summary for both operations).
 *
 * The first 15 arguments, their layouts and errors are indexer_q_prep_bf16's;
 * x2, M2, K2, ldx2, q2, ldq2, scales2, s_stride_m2, s_stride_w2 are
 * fp8_quant_1x128_ue8m0's (x, M, K, ldx, q, ldq, scales, s_stride_m,
 * s_stride_w), with the same checks and M2 at most 256 (else
 * IQP_ERR_UNSUPPORTED). Both outputs are byte for byte those of the two
 * separate calls. M2 == 0 or K2 == 0: the first call alone; M == 0: the
 * quantization alone (its own launch). The x2 / q2 / scales2 regions must
 * not overlap the other call's buffers.
 */
int indexer_q_prep_bf16_with_quant(const void* x, int64_t ldx, const void* w, int64_t ldw,
                                   const uint8_t* w_scales,
                                   int64_t M, int64_t K, int32_t H, int32_t D, int32_t rope_dim,
                                   const int64_t* positions, const float* cos_sin, int64_t max_pos,
                                   uint8_t* q_fp4, uint8_t* q_scales,
                                   const void* x2, int64_t M2, int64_t K2, int64_t ldx2,
                                   void* q2, int64_t ldq2, int32_t* scales2,
                                   int64_t s_stride_m2, int64_t s_stride_w2,
                                   void* stream);

/*
 * indexer_q_workspace_bytes — bytes of the workspace that
 * indexer_q_prep_bf16_with_quant_ws needs for H heads: 256 bytes of counters
 * per 32 heads (rounded up), then 64 KiB per head of float32 partial sums.
 * 4,194,816 bytes at H = 64. H <= 0: 0. (A workspace of B bytes keeps its
 * counters for the most heads it can hold, B / 65544, so one workspace
 * serves calls with any head count it is large enough for.)
 */
int64_t indexer_q_workspace_bytes(int32_t H);

/*
 * indexer_q_prep_bf16_with_quant_ws — indexer_q_prep_bf16_with_quant with a
 * workspace (the same arguments, then workspace, workspace_bytes). From 12
 * to 64 tokens the one-launch kernel then splits each head's K range (12
 * blocks of 128) over 3 workgroups (12 to 32 tokens) or 2 (33 to 64): each
 * quantizes only its blocks of X and streams only its blocks of W, stores
 * its float32 partial sums in the workspace and takes a ticket from the head
 * and tile's counter there; the workgroup that draws the last ticket adds the
 * partial sums in split order, resets the counter and runs the RoPE /
 * Hadamard / FP4 epilogue. Outside that range the workspace is not touched.
 * The GEMM is the same block-scaled FP8 contraction as in the unsplit kernel
 * (TensorRT-LLM PR "Fuse DeepSeek-V4 Indexer Q projection with CuTe DSL",
 * sequence diagram); only the order in which the float32 partial sums are
 * added differs, and it is fixed, so results are deterministic. Measured on
 * MI355X with an [M, 7168] quantization beside it, weights in the Infinity
 * Cache: 7.9 us against 8.6 at 24 tokens, 8.2 against 9.5 at 32, 8.7
 * against 9.6 at 48; weights in HBM: 8.7 against 9.9 at 16 tokens, 9.1
 * against 11.6 at 32.
 *
 * workspace: device memory of at least indexer_q_workspace_bytes(H) bytes,
 * 256-byte aligned, owned by the caller, filled with zeros before its first
 * use (each call leaves its counters at zero again; the partial sums need no
 * clearing). Calls that share a workspace must not run concurrently (one
 * workspace per stream, or order the calls): their counters would mix.
 *
 * Errors: null workspace or workspace_bytes too small: IQP_ERR_INVALID;
 * workspace not 256-byte aligned: IQP_ERR_UNSUPPORTED; everything else as in
 * indexer_q_prep_bf16_with_quant.
 */
int indexer_q_prep_bf16_with_quant_ws(const void* x, int64_t ldx, const void* w, int64_t ldw,
                                      const uint8_t* w_scales,
                                      int64_t M, int64_t K, int32_t H, int32_t D, int32_t rope_dim,
                                      const int64_t* positions, const float* cos_sin, int64_t max_pos,
                                      uint8_t* q_fp4, uint8_t* q_scales,
                                      const void* x2, int64_t M2, int64_t K2, int64_t ldx2,
                                      void* q2, int64_t ldq2, int32_t* scales2,
                                      int64_t s_stride_m2, int64_t s_stride_w2,
                                      void* workspace, int64_t workspace_bytes, void* stream);

/*
 * indexer_q_prep_bf16_with_quant_noalloc — indexer_q_prep_bf16_with_quant_ws
 * for callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation): the same
 * arguments without the workspace, which is instead the library's own
 * scratch, a static device array of indexer_q_workspace_bytes(
 * IQP_NOALLOC_MAX_HEADS) = 4,194,816 bytes that each GPU the library runs on
 * holds until the process ends (it is zero when the library is loaded, and
 * every call leaves its counters at zero). The call allocates nothing.
 *
 * Every call on one GPU shares that GPU's scratch: calls that overlap on one
 * GPU (on different streams, or from several threads) race and must not be
 * made; order them on one stream. Results are byte for byte those of
 * indexer_q_prep_bf16_with_quant_ws.
 *
 * Errors: H > IQP_NOALLOC_MAX_HEADS: IQP_ERR_UNSUPPORTED (the scratch is too
 * small; use indexer_q_prep_bf16_with_quant_ws); otherwise as in
 * indexer_q_prep_bf16_with_quant (the scratch's address is looked up once per
 * device, at the first call that gets past the checks; IQP_ERR_HIP if that
 * fails).
 */
#define IQP_NOALLOC_MAX_HEADS 64
int indexer_q_prep_bf16_with_quant_noalloc(const void* x, int64_t ldx, const void* w, int64_t ldw,
                                           const uint8_t* w_scales,
                                           int64_t M, int64_t K, int32_t H, int32_t D, int32_t rope_dim,
                                           const int64_t* positions, const float* cos_sin, int64_t max_pos,
                                           uint8_t* q_fp4, uint8_t* q_scales,
                                           const void* x2, int64_t M2, int64_t K2, int64_t ldx2,
                                           void* q2, int64_t ldq2, int32_t* scales2,
                                           int64_t s_stride_m2, int64_t s_stride_w2, void* stream);

/*
 * indexer_q_rope_hadamard_fp4 — the epilogue of indexer_q_gemm_rope_fp4 as a
 * standalone launch over a bf16 Q: RoPE + Hadamard-128 + FP4 e2m1.
 *
 * TensorRT-LLM PR "Fuse DeepSeek-V4 Indexer Q projection with CuTe DSL",
 * Description / Paths compared (the unfused chain: the Q GEMM writes a bf16
 * Q, then an in-place RoPE kernel and an FP4 quantization kernel with scale
 * copies run on it); tokenspeed PR "perf(deepseek-v4): accelerate indexer Q
 * and packed FP8 quantization", Summary (the RoPE kernel, the Hadamard
 * transform and the fused FP4 cat kernel of the Q preparation).
 *
 * For every token m and head h, with Q_d = q[m * ldq + 128 h + d] widened to
 * float32, the RoPE, Hadamard and FP4 steps are those of
 * indexer_q_gemm_rope_fp4 (same table, same output layout and rounding)
 * when flags is 0. flags may select convention variants:
 *   IQP_ROPE_INTERLEAVED      pair i (angle row entries i and rope_dim/2 + i of
 *                             the table, as before) is dims (2i, 2i + 1);
 *   IQP_FP4_SCALE_OCP_FLOOR   e = floor(log2 max(amax, 1e-4)) - 2 (so e >= -16),
 *                             codes = E2M1 RNE of z * 2^-e saturated at +-6.
 * Other bits: IQP_ERR_INVALID.
 *
 *   q          bf16 [M, H*D], row stride ldq (elements, >= H*D); 16-byte
 *              aligned and ldq a multiple of 8, else IQP_ERR_UNSUPPORTED.
 *              Read only (no in-place RoPE).
 *   M          tokens (>= 0); H >= 1; D must be 128 and rope_dim 64 (else
 *              IQP_ERR_UNSUPPORTED); M < 2^31 and H <= 64 * 65535.
 *   positions  int64 [M]; outside [0, max_pos) is a precondition violation,
 *              clamped into range as in indexer_q_gemm_rope_fp4.
 *   cos_sin    float32 [max_pos, rope_dim] as in indexer_q_gemm_rope_fp4,
 *              16-byte aligned; max_pos >= 1.
 *   q_fp4      uint8 [M, H, D/2] packed E2M1 codes, 16-byte aligned.
 *   q_scales   uint8 [M, H, D/32] UE8M0 bytes, 4-byte aligned.
 *
 * Q must be finite.
 */
int indexer_q_rope_hadamard_fp4(const void* q, int64_t ldq, int64_t M, int32_t H, int32_t D,
                                int32_t rope_dim, const int64_t* positions,
                                const float* cos_sin, int64_t max_pos,
                                uint8_t* q_fp4, uint8_t* q_scales, int32_t flags, void* stream);

/*
 * fp8_quant_weight_128x128_ue8m0 — weight preparation: bf16 weights to the
 * E4M3 codes and per-tile UE8M0 scales that indexer_q_gemm_rope_fp4 and
 * indexer_q_prep_bf16 take as w / w_scales. Not on the per-token path: it
 * runs when weights are loaded or updated.
 *
 * The pages only say the Q projection is a block-scaled FP8 GEMM (tokenspeed
 * PR "perf(deepseek-v4): accelerate indexer Q and packed FP8 quantization",
 * Summary; TensorRT-LLM PR "Fuse DeepSeek-V4 Indexer Q projection with CuTe
 * DSL", sequence diagram); the weight format is a reading: one scale per
 * 128x128 tile, chosen like the activations' scales. For every tile (a, b):
 *   amax = max(max |w| over rows 128a.., columns 128b.., 1e-4)
 *   e    = ceil(log2(amax / 448)) exact;  scales[a * ld_scales + b] = e + 127
 *   q    = E4M3 round-to-nearest-even of w * 2^-e (never saturates)
 *
 *   w          bf16 [N, K], row stride ldw (elements, >= K); 16-byte aligned,
 *              ldw a multiple of 8.
 *   q          E4M3 bytes [N, K], row stride ldq (bytes, >= K); 8-byte
 *              aligned, ldq a multiple of 8.
 *   scales     uint8 [N/128, K/128], row stride ld_scales (bytes, >= K/128).
 *   N, K       multiples of 128 (else IQP_ERR_UNSUPPORTED); N/128 <= 65535.
 * Inputs must be finite.
 */
int fp8_quant_weight_128x128_ue8m0(const void* w, int64_t N, int64_t K, int64_t ldw,
                                   void* q, int64_t ldq, uint8_t* scales, int64_t ld_scales,
                                   void* stream);

/*
 * iqp_rope_cos_sin_table — builds the standard RoPE table that
 * indexer_q_gemm_rope_fp4 reads: for 0 <= p < max_pos and i < rope_dim/2,
 *   cos_sin[p, i] = cos(p * theta^(-2i/rope_dim)),
 *   cos_sin[p, rope_dim/2 + i] = sin(p * theta^(-2i/rope_dim)),
 * evaluated in float64 on the device and rounded to float32 once.
 * (tokenspeed PR "perf(deepseek-v4): accelerate indexer Q and packed FP8
 * quantization", Summary: RoPE on the indexer Q; the base and layout are not
 * on the page, theta = 10000 is the usual base.)
 *
 *   cos_sin   float32 [max_pos, rope_dim], 4-byte aligned. rope_dim even, > 0;
 *             theta > 0; max_pos >= 0 (0: no-op).
 */
int iqp_rope_cos_sin_table(double theta, int64_t max_pos, int32_t rope_dim,
                           float* cos_sin, void* stream);

/*
 * iqp_rope_table_lanes — the lane-ordered copy of a RoPE table that
 * indexer_q_gemm_rope_fp4_lanes reads (the same values, rearranged; built
 * once per table). Element k = 2048 b + 256 L + 4 (2 r + h) + e holds
 *   cos_sin[32 b + r, 32 (L % 2) + 8 (L / 2) + 4 h + e]
 * for 0 <= L < 8, 0 <= r < 32, h < 2, e < 4 where 32 b + r < max_pos, and 0.0
 * past max_pos: block b holds positions 32 b .. 32 b + 31, each 16-byte
 * piece the load one kernel lane makes. (tokenspeed PR "perf(deepseek-v4):
 * accelerate indexer Q and packed FP8 quantization", Summary: RoPE on the
 * indexer Q; the layout is this library's.)
 *
 *   cos_sin  float32 [max_pos, rope_dim], 16-byte aligned; rope_dim must be
 *            64 (else IQP_ERR_UNSUPPORTED).
 *   out      float32, ceil(max_pos / 32) * 2048 elements, 16-byte aligned;
 *            must not overlap cos_sin.
 *   max_pos >= 0 (0: no-op).
 */
int iqp_rope_table_lanes(const float* cos_sin, int64_t max_pos, int32_t rope_dim,
                         float* out, void* stream);

/*
 * iqp_debug_indexer_q_f32 — diagnostic twin of indexer_q_gemm_rope_fp4 for
 * parity testing of its stages (TensorRT-LLM PR "Fuse DeepSeek-V4 Indexer Q
 * projection with CuTe DSL", sequence diagram: the GEMM result feeds the
 * RoPE / FP4 epilogue): same inputs, but instead of FP4 codes it writes
 * float32 out[M, H*D] holding
 *   stage 0: Q (the GEMM output),
 *   stage 1: Q after RoPE,
 *   stage 2: z (after RoPE and the normalized Hadamard rotation),
 * all three from the general fused kernel (every supported shape), or
 *   stage 3: Q from the K loop of the kernel indexer_q_gemm_rope_fp4 runs
 *            for these arguments (the small-batch, pipelined or split-role
 *            kernel, built with its epilogue replaced by a float32 store; the
 *            general kernel's stage 0 where that is the kernel it runs).
 * out is 16-byte aligned; any other stage is IQP_ERR_INVALID.
 */
int iqp_debug_indexer_q_f32(const void* a, int64_t lda,
                            const int32_t* a_scales, int64_t as_stride_m, int64_t as_stride_w,
                            const void* w, int64_t ldw,
                            const uint8_t* w_scales,
                            int64_t M, int64_t K, int32_t H, int32_t D, int32_t rope_dim,
                            const int64_t* positions,
                            const float* cos_sin, int64_t max_pos,
                            float* out, int32_t stage,
                            void* stream);

/*
 * iqp_debug_indexer_q_prep_bf16_f32 — diagnostic twin of indexer_q_prep_bf16
 * (same pages, same arguments and limits): the one-launch kernel, quantizing
 * x itself, with its epilogue replaced by a float32 store of Q (the GEMM
 * output) to out[M, H*D], 16-byte aligned.
 */
int iqp_debug_indexer_q_prep_bf16_f32(const void* x, int64_t ldx, const void* w, int64_t ldw,
                                      const uint8_t* w_scales,
                                      int64_t M, int64_t K, int32_t H, int32_t D, int32_t rope_dim,
                                      const int64_t* positions, const float* cos_sin, int64_t max_pos,
                                      float* out, void* stream);

/*
 * iqp_debug_indexer_q_clock — indexer_q_gemm_rope_fp4 (same arguments, same
 * q_fp4 / q_scales bytes) from a build of its kernel that also records the
 * shader clock, for reading measured throughput against the clock the chip
 * ran at (tokenspeed PR "perf(deepseek-v4): accelerate indexer Q and packed
 * FP8 quantization", Performance: the pages quote kernel times with no
 * clock). Supported where the call runs the split-role kernel (K = 1536,
 * 257 tokens or more); elsewhere IQP_ERR_UNSUPPORTED with nothing enqueued.
 *
 *   cos_sin_lanes   NULL (the build that reads cos_sin), or the table's
 *                   lane-ordered copy as indexer_q_gemm_rope_fp4_lanes takes
 *                   it (the build that reads that; 16-byte aligned).
 *
 *   stamps          uint64 [4 * workgroups], 16-byte aligned: for workgroup
 *                   g, stamps[4g], [4g+1] = the shader clock counter
 *                   (s_memtime) at its start and end, [4g+2], [4g+3] = the
 *                   constant-rate counter (s_memrealtime, ticking at the
 *                   wall clock rate of iqp_device_clock_rates) at the same
 *                   points; all four 0 for a workgroup given no tokens.
 *   stamp_capacity  elements of stamps; below 4 * workgroups: IQP_ERR_INVALID,
 *                   nothing enqueued.
 *   n_workgroups    host pointer, set to the launch's workgroup count before
 *                   any other check of the stamps (0 when unsupported or
 *                   invalid otherwise).
 * Mean shader clock of a workgroup = (end - start of s_memtime) / (end -
 * start of s_memrealtime) * wall clock rate.
 */
int iqp_debug_indexer_q_clock(const void* a, int64_t lda,
                              const int32_t* a_scales, int64_t as_stride_m, int64_t as_stride_w,
                              const void* w, int64_t ldw,
                              const uint8_t* w_scales,
                              int64_t M, int64_t K, int32_t H, int32_t D, int32_t rope_dim,
                              const int64_t* positions,
                              const float* cos_sin, const float* cos_sin_lanes, int64_t max_pos,
                              uint8_t* q_fp4, uint8_t* q_scales,
                              uint64_t* stamps, int64_t stamp_capacity, int64_t* n_workgroups,
                              void* stream);

/*
 * iqp_device_clock_rates — the current device's constant-rate counter
 * frequency (the rate of iqp_debug_indexer_q_clock's realtime stamps) and its
 * peak shader clock, in Hz, into two host int64 values. IQP_ERR_HIP if the
 * runtime cannot report them.
 */
int iqp_device_clock_rates(int64_t* wall_clock_hz, int64_t* peak_shader_clock_hz);

/*
 * fp8_gemm_1x128_128x128 — block-scaled FP8 matrix product, bf16 out: the
 * layer's other projections, on the operands of fp8_quant_1x128_ue8m0 and
 * fp8_quant_weight_128x128_ue8m0.
 *
 *   out[m, n] = bf16( sum_j 2^(ea(m,j) + ew(n/128,j)) sum_{k in block j} A[m,k] W[n,k] )
 * (float32 accumulation, one rounding to bf16). Within 64 columns the matrix cores
 * add products at a fixed precision below the largest of them: such a sum is off by
 * about 2^-11.3 of that product at most (measured), usually by 2^-14.5.
 *
 *   a, lda, a_scales, as_stride_m, as_stride_w, w, ldw   as in
 *              indexer_q_gemm_rope_fp4, with row strides that are multiples
 *              of 16 up to 2^22, as_stride_m below 2^19 and as_stride_w below
 *              2^27 / ceil(K/512); K a multiple of 128, at most 32768.
 *   w          E4M3 [N, K]; N is any (the scales' last tile may be partial).
 *   w_scales   UE8M0 [ceil(N/128), K/128], row stride ld_ws (bytes, >= K/128).
 *   out        bf16 [M, N], row stride ldo (elements, >= N), 2-byte aligned
 *              (16-byte stores where it is 16-byte aligned and ldo a multiple
 *              of 8). Must not overlap the inputs.
 *   workspace  NULL, or fp8_gemm_workspace_bytes(M, N, K) bytes of device
 *              memory, 256-byte aligned: with it a product of few output tiles
 *              and many K blocks is split over K (two launches). Its contents do
 *              not matter before and mean nothing after; calls that share one
 *              must not overlap. Where that size is 0 it is not used (also for
 *              sizes that the product refuses).
 * M == 0 or N == 0: no-op. The sum must fit float32, as there. The order in
 * which K blocks are added depends on M, N, K and the workspace's presence only.
 */
int64_t fp8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);
int fp8_gemm_1x128_128x128(const void* a, int64_t lda,
                           const int32_t* a_scales, int64_t as_stride_m, int64_t as_stride_w,
                           const void* w, int64_t ldw, const uint8_t* w_scales, int64_t ld_ws,
                           int64_t M, int64_t N, int64_t K, void* out, int64_t ldo,
                           void* workspace, int64_t workspace_bytes, void* stream);

/*
 * iqp_debug_fp8_gemm_kernel — the name of the kernel that
 * fp8_gemm_1x128_128x128 takes for these sizes, with a workspace or without
 * ("stream 32x16", "tile 256x256": weight rows x tokens of a workgroup), "" for
 * sizes that it refuses. Static storage; touches no device. For tests that mean
 * to reach each of them.
 */
const char* iqp_debug_fp8_gemm_kernel(int64_t M, int64_t N, int64_t K, int32_t with_workspace);

/*
 * qk_norm_rope — RMS norm of every query and key head, times its weights,
 * then RoPE, in one pass.
 *
 * For every token m and head x of D values (queries with q_weight, keys with
 * k_weight), in float32 with one rounding to bf16:
 *   y_d = x_d / sqrt(mean(x^2) + eps) * weight_d
 *   RoPE on dims [0, rope_dim) with the row positions[m] of cos_sin: pairs
 *   (i, i + rope_dim/2), or with IQP_ROPE_INTERLEAVED (2i, 2i + 1), as in
 *   indexer_q_rope_hadamard_fp4.
 *
 *   q, k       bf16 [M, Hq*D] and [M, Hk*D], row strides ldq, ldk (elements):
 *              16-byte aligned, strides multiples of 8.
 *   q_out, k_out   likewise, strides ldqo, ldko; may be q and k themselves (same
 *              strides), otherwise must not overlap them.
 *   q_weight, k_weight   bf16 [D], 16-byte aligned, finite.
 *   D          64, 128 or 256; rope_dim a multiple of 16, 16 to D; eps >= 0.
 *   positions, cos_sin, max_pos   as in indexer_q_gemm_rope_fp4 (table of
 *              rope_dim columns; positions outside it are clamped).
 *   flags      0 or IQP_ROPE_INTERLEAVED, else IQP_ERR_INVALID.
 */
int qk_norm_rope(const void* q, int64_t ldq, const void* k, int64_t ldk, int64_t M, int32_t Hq, int32_t Hk,
                 int32_t D, int32_t rope_dim, const void* q_weight, const void* k_weight, float eps,
                 const int64_t* positions, const float* cos_sin, int64_t max_pos,
                 void* q_out, int64_t ldqo, void* k_out, int64_t ldko, int32_t flags, void* stream);

/*
 * The FP8 key/value cache of one layer: n_blocks blocks of block_size tokens
 * (16, 32, 64 or 128), Hk key heads of D values (64 or 128):
 *   k_cache   E4M3 [n_blocks, Hk, block_size, D]
 *   v_cache   E4M3 [n_blocks, Hk, D, block_size] (a dim's tokens together, the
 *             order in which attention multiplies them)
 *   k_scales, v_scales   UE8M0 [n_blocks, Hk]: value = code * 2^(byte - 127)
 * k_cache and v_cache 16-byte aligned. All contiguous.
 *
 * A batch of S sequences and T rows: rows cu_rows[s] .. cu_rows[s+1] - 1 are
 * the last tokens of sequence s, which has seq_lens[s] tokens with them (row
 * cu_rows[s] + i is position seq_lens[s] - (cu_rows[s+1] - cu_rows[s]) + i).
 *   cu_rows      int32 [S + 1], non-decreasing; values outside [0, T] are
 *                clamped into it. Rows before cu_rows[0] and from cu_rows[S]
 *                on belong to no sequence: they are not read, nor written.
 *   seq_lens     int32 [S].
 *   block_table  int32 [S, max_blocks], row stride ld_table: position p of
 *                sequence s is token p % block_size of block
 *                block_table[s, p / block_size]. An entry outside [0,
 *                n_blocks), a position of max_blocks * block_size or more (at
 *                most 2^30), and a position below 0 mean a token that is not held.
 * These three arrays are read on the device: a call can be captured once and
 * replayed with other lengths, up to the T rows and S sequences it was given.
 * T == 0 or S == 0: no-op.
 */

/*
 * kv_cache_append_fp8 — quantise new keys and values into the cache.
 *
 * For each block and head that rows of the batch fall into, with lo the first
 * such token of the block and amax taken over those rows' values in it:
 *   need = max(ceil(log2(amax / 448)), -22)            (the 1x128 quantizer's rule)
 *   e    = need where lo == 0, else max(need, byte - 127)
 *   code = E4M3 round-to-nearest-even of x * 2^-e;     byte = e + 127
 * Where e > byte - 127 before the call, the codes of the block's tokens
 * 0 .. lo - 1 become E4M3 RNE of code * 2^(byte - 127 - e). Tokens behind the
 * last one written keep their codes (a sequence ends with the rows it is
 * given). Rows that are not held are left out.
 *
 *   k, v       bf16 [T, Hk*D], row strides ldk, ldv (elements); 16-byte
 *              aligned, strides multiples of 8. Finite.
 * No block may be named by two of the table entries that a call's rows fall
 * into, of two sequences or of one.
 */
int kv_cache_append_fp8(const void* k, int64_t ldk, const void* v, int64_t ldv, int64_t T, int32_t Hk, int32_t D,
                        void* k_cache, void* v_cache, uint8_t* k_scales, uint8_t* v_scales,
                        int64_t n_blocks, int32_t block_size,
                        const int32_t* block_table, int64_t ld_table, int32_t max_blocks,
                        const int32_t* seq_lens, const int32_t* cu_rows, int32_t S, void* stream);

/*
 * kv_cache_read_fp8 — the batch's rows read back from the cache as bf16
 * (exact: a code has 4 significant bits).
 *
 *   k_out, v_out   bf16 [T, Hk*D], row strides ldk, ldv (elements); 16-byte
 *                  aligned, strides multiples of 8. Rows of tokens that are not
 *                  held, and rows behind cu_rows[S], are left as they were.
 */
int kv_cache_read_fp8(const void* k_cache, const void* v_cache, const uint8_t* k_scales, const uint8_t* v_scales,
                      int64_t n_blocks, int32_t block_size, int32_t Hk, int32_t D,
                      const int32_t* block_table, int64_t ld_table, int32_t max_blocks,
                      const int32_t* seq_lens, const int32_t* cu_rows, int32_t S,
                      void* k_out, int64_t ldk, void* v_out, int64_t ldv, int64_t T, void* stream);

/*
 * attention_fp8_kv — causal attention of bf16 queries over the FP8 cache.
 *
 * For the row at position p of a sequence and query head h, over the held
 * tokens t <= p (and t > p - window where window > 0, up to 2^31 - 1) of key head h / (Hq / Hk):
 *   out = sum_t w_t v_t / sum_t w_t,  w_t = exp(scale * q . k_t)
 * with k_t, v_t the values the cache stands for; zeros where there is no such
 * token. Scores, maxima and sums are float32. For the second product the weights
 * are rounded to fp16 relative to the row's largest w_t 2^e_t (e_t the value
 * exponent of t's block): each is off by at most 2^-11 of itself, and those below
 * 2^-21 of the largest by at most 2^-32 of the largest. The latter moves the output
 * of a row that sees n tokens by at most n 2^-31 times the largest value of the
 * block of the largest w_t 2^e_t (an eighth of bf16's own half step at a million
 * tokens of like sizes). The value exponents that a row sees may lie up to 100
 * apart (always so where no value written exceeds 2^86), and must not lie below
 * -80 (what kv_cache_append_fp8 writes does not lie below -22): beyond that weights
 * are lost from the sum.
 *
 *   q, out     bf16 [T, Hq*D], row strides ldq, ldo (elements); 16-byte
 *              aligned, strides multiples of 8; out must not overlap q. Rows
 *              behind cu_rows[S] are left as they were. A row of q that holds a NaN
 *              or an infinity makes no other row's output NaN.
 *   k_cache, v_cache   held tokens' codes other than NaN (kv_cache_append_fp8 writes
 *              none for finite values): a NaN among the values of a token reaches
 *              rows computed beside those that see it, also ones before it. What
 *              lies in blocks that are not held, behind a sequence and before every
 *              window does not matter.
 *   Hq         a multiple of Hk (else IQP_ERR_INVALID).
 *   scale      2^-64 to 2^64 (else IQP_ERR_INVALID); times the power of two of a
 *              key scale it must lie between 2^-100 and 2^126.
 *   workspace  attention_fp8_kv_workspace_bytes(D) bytes of device memory,
 *              256-byte aligned; its contents do not matter before and mean
 *              nothing after. Calls that share one must not overlap.
 * The same call gives the same bits. The order of its sums depends on T, S, Hq,
 * Hk, D, the table's width and the window, and a row's weights are rounded relative
 * to a maximum that rows computed beside it share in raising, so a row's last bit
 * may differ between batches.
 */
int64_t attention_fp8_kv_workspace_bytes(int32_t D);
int attention_fp8_kv(const void* q, int64_t ldq, int64_t T, int32_t Hq, int32_t Hk, int32_t D,
                     const void* k_cache, const void* v_cache, const uint8_t* k_scales, const uint8_t* v_scales,
                     int64_t n_blocks, int32_t block_size,
                     const int32_t* block_table, int64_t ld_table, int32_t max_blocks,
                     const int32_t* seq_lens, const int32_t* cu_rows, int32_t S,
                     float scale, int32_t window, void* out, int64_t ldo,
                     void* workspace, int64_t workspace_bytes, void* stream);

/*
 * moe_route — the top_k experts of every token and their weights.
 *
 * With z the logits of a token, and
 *   p_e = exp(z_e) / sum_f exp(z_f)      IQP_SCORE_SOFTMAX
 *         1 / (1 + exp(-z_e))            IQP_SCORE_SIGMOID
 *         sqrt(log(1 + exp(z_e)))        IQP_SCORE_SQRT_SOFTPLUS
 * the experts are the first top_k in falling order of z_e, or with a bias of
 * p_e + bias_e, the lower index first where these are equal, and
 *   weight = scale * p_e / (sum of p over the chosen ones if renormalize, else 1).
 * All in float64 and rounded to float32 once. Logits are compared exactly, sums p_e +
 * bias_e by their first 42 mantissa bits, and count as equal where these agree: a
 * rounding of an exponential shows in the choice only where a sum lies within a few
 * units of its last, 52nd bit from where those 42 change. A token's results do not
 * depend on what other tokens hold; how many there are decides between kernels that
 * add the chosen scores, and form a sigmoid, in ways that differ in float64's last
 * bits. An expert whose logit is -inf comes after all others and has weight 0; a token
 * all of whose logits are -inf gets experts 0 .. top_k - 1 with weights 0. A NaN logit
 * comes before all others; it, and +inf under IQP_SCORE_SOFTMAX, make weights of the
 * token NaN, of other tokens none, and where p_e + bias_e is NaN the logits order the
 * experts, which are distinct and in range whatever the logits hold.
 *
 *   logits   float32, or bf16 where logits_bf16 is not 0, [M, E], row stride ld
 *            (elements, >= E); 4- or 2-byte aligned. E 1 to 1024, M up to 2^26 - 4.
 *   bias     NULL, or float32 [E], finite.
 *   top_k    1 to min(E, 64).
 *   weights  float32 [M, top_k];  experts  int32 [M, top_k]; both contiguous.
 */
#define IQP_SCORE_SOFTMAX        0
#define IQP_SCORE_SIGMOID        1
#define IQP_SCORE_SQRT_SOFTPLUS  2
int moe_route(const void* logits, int64_t ld, int32_t logits_bf16, const float* bias, int64_t M, int32_t E,
              int32_t top_k, int32_t scoring, int32_t renormalize, float scale, float* weights, int32_t* experts,
              void* stream);

/*
 * group_rows — the R entries of index sorted by group, entries of a group in
 * their own order: group g has the places offsets[g] .. offsets[g+1] - 1, place
 * i holds entry rows[i], entry r is at place slots[r]. An entry outside [0, G)
 * is in no group: its slot is -1, and rows holds -1 from offsets[G] on.
 *
 *   index      int32 [R]: moe_route's experts [M, top_k], or an adapter a token.
 *   offsets    int32 [G + 1];  rows, slots  int32 [R]. G 1 to 1024. None may overlap
 *              another or index.
 *   workspace  group_rows_workspace_bytes(R, G) bytes of device memory, 4-byte
 *              aligned (NULL where that is 0); its contents do not matter before
 *              and mean nothing after. Calls that share one must not overlap.
 * R == 0: offsets are all 0.
 */
int64_t group_rows_workspace_bytes(int64_t R, int32_t G);
int group_rows(const int32_t* index, int64_t R, int32_t G, int32_t* offsets, int32_t* rows, int32_t* slots,
               void* workspace, int64_t workspace_bytes, void* stream);

/*
 * fp8_grouped_gemm_1x128_128x128 — fp8_gemm_1x128_128x128 with weights of its own
 * for every group of rows, over places sorted by group (group_rows): for place i
 * of group g
 *   out[i, n] = bf16( sum_j 2^(ea(src,j) + ew(g,n/128,j)) sum_{k in block j} A[src,k] W[g,n,k] )
 * with src = i where top_k is 0 (M == R), else rows[i] / top_k, the token that the
 * place's entry belongs to (M * top_k == R). Rounding and accuracy as there.
 *
 * fp8_grouped_swiglu_1x128 — the same product with 2 I weight rows, gates 0 ..
 * I - 1 and ups I .. 2 I - 1, then for channel c
 *   h[i, c] = y_c / (1 + exp(-y_c)) * y_(I+c)       (float32, y not rounded before)
 * quantised from float32 as fp8_quant_1x128_ue8m0 quantises bf16: for each 128
 * channels e = max(ceil(log2(amax / 448)), -22), codes E4M3 RNE of h 2^-e.
 *
 *   a, lda, a_scales, as_stride_m, as_stride_w   as in fp8_gemm_1x128_128x128, M
 *              rows; they and their scale words each reach less than 2^31 bytes.
 *   w          E4M3 [G, N, K] (swiglu: [G, 2 I, K]), strides ldwg, ldw (bytes,
 *              multiples of 16, ldw up to 2^22), 16-byte aligned. w_scales UE8M0 [G,
 *              ceil(N/128), K/128], strides ld_wsg, ld_ws (bytes).
 *   offsets, rows, R, G   group_rows' (rows may be NULL where top_k is 0). Read on
 *              the device; offsets outside [0, R] are clamped into it, rows that
 *              name no token read zeros. Places in no group are not computed.
 *   K          a multiple of 128, at most 32768;  I  a multiple of 128;  N  any.
 *   out        bf16 [R, N], row stride ldo (elements, >= N), 2-byte aligned (fastest
 *              where 16-byte aligned with ldo a multiple of 8).
 *   q          E4M3 [R, I], row stride ldq (bytes, a multiple of 16), 16-byte
 *              aligned; q_scales packed words [R, ceil(I/512)] in either layout of
 *              fp8_quant_1x128_ue8m0.
 *              Rows of no group are left as they were in all three, and none of them
 *              may overlap the inputs. (R / 256 + min(G, R)) ceil(N / 256) below 2^24 -
 *              256, N being 2 I for swiglu.
 * R == 0, N == 0 or I == 0: no-op. The results must be finite in float32. The same
 * call gives the same bits; how many rows a place's group has, and for up to 16 of
 * them the group's number, decide in which order its sums are added, and so its last
 * bit.
 */
int fp8_grouped_gemm_1x128_128x128(const void* a, int64_t lda, const int32_t* a_scales, int64_t as_stride_m,
                                   int64_t as_stride_w, int64_t M, const void* w, int64_t ldwg, int64_t ldw,
                                   const uint8_t* w_scales, int64_t ld_wsg, int64_t ld_ws, const int32_t* offsets,
                                   const int32_t* rows, int64_t R, int32_t G, int32_t top_k, int64_t N, int64_t K,
                                   void* out, int64_t ldo, void* stream);
int fp8_grouped_swiglu_1x128(const void* a, int64_t lda, const int32_t* a_scales, int64_t as_stride_m,
                             int64_t as_stride_w, int64_t M, const void* w, int64_t ldwg, int64_t ldw,
                             const uint8_t* w_scales, int64_t ld_wsg, int64_t ld_ws, const int32_t* offsets,
                             const int32_t* rows, int64_t R, int32_t G, int32_t top_k, int64_t I, int64_t K,
                             void* q, int64_t ldq, int32_t* q_scales, int64_t qs_stride_m, int64_t qs_stride_w,
                             void* stream);

/*
 * moe_combine — every token's weighted sum of its experts' rows:
 *   out[m] = bf16( sum_j weights[m, j] y[slots[m, j]] + shared[m] )
 * summed in float32 in the order of j. Slots outside [0, R) are left out (an
 * expert that is not held here); a token without any gives shared's row, or zeros.
 *
 *   y        bf16 [R, d], row stride ldy;  shared  NULL, or bf16 [M, d], row stride
 *            ld_shared;  out  bf16 [M, d], row stride ldo, may be shared itself
 *            (same stride), otherwise must not overlap the inputs. 16-byte aligned,
 *            d and the strides multiples of 8; M ceil(d / 2048) below 2^24.
 *   slots    int32 [M, top_k];  weights  float32 [M, top_k]; contiguous. top_k >= 1.
 */
int moe_combine(const void* y, int64_t ldy, int64_t R, const int32_t* slots, const float* weights, int64_t M,
                int32_t top_k, int64_t d, const void* shared, int64_t ld_shared, void* out, int64_t ldo, void* stream);

/*
 * lora_add — low-rank adapters of many requests, added in place to the output of
 * the projection that they share: for every place i of group g, with m = rows[i],
 *   out[m] = bf16( out[m] + scales[g] * B[g] (A[g] x[m]) )
 * (float32 sums; A[g] x[m] goes into the second product as two bf16 parts, 16
 * significant bits, an infinite one as itself). Rows in no group keep their bits.
 *
 *   x          bf16 [M, K], row stride ldx; 16-byte aligned, K and ldx multiples of 8, K
 *              at most 2^22; it reaches less than 2^31 bytes.
 *   a, b       bf16 [G, rank, K] and [G, N, rank], contiguous, 16-byte aligned, finite;
 *              rank a multiple of 8, 8 to 128 (adapters of a lower one: zeros).
 *   scales     NULL (1), or float32 [G].
 *   offsets, rows, G   group_rows' of one adapter a token (R = M). Read on the device;
 *              offsets outside [0, M] are clamped, rows outside [0, M) left out. No
 *              row may be at two places (group_rows gives none).
 *   out        bf16 [M, N], row stride ldo, 2-byte aligned (fastest where 16-byte
 *              aligned with ldo a multiple of 8). Must not overlap the others. (M / 64 +
 *              min(G, M)) ceil(N / 256) below 2^24 - 8.
 *   workspace  lora_add_workspace_bytes(M, G, rank, K) bytes of device memory (0 for an
 *              M, G, rank or K that is refused), 256-byte aligned; its contents do not
 *              matter before and mean nothing after. Calls that share one must not overlap.
 * M == 0, N == 0 or G == 0: no-op. The same call gives the same bits.
 */
int64_t lora_add_workspace_bytes(int64_t M, int32_t G, int32_t rank, int64_t K);
int lora_add(const void* x, int64_t ldx, int64_t M, int64_t K, const void* a, const void* b, const float* scales,
             int32_t rank, const int32_t* offsets, const int32_t* rows, int32_t G, int64_t N, void* out, int64_t ldo,
             void* workspace, int64_t workspace_bytes, void* stream);

/* Human-readable name of a status code (static storage; never NULL). */
const char* iqp_status_string(int status);

/* IQP_ABI_VERSION of the built library. */
int iqp_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* IQPREP_H */
