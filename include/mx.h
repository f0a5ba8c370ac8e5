/*
 * mx.h - C ABI of the inline-quantized A4W4 MXFP4 GEMM library for MI355X (gfx950).
 *
 * The operation ("[gfx950][FlyDSL] Add direct dense A4W4 MXFP4 GEMM", Summary and
 * Implementation): BF16 activations A[M,K] are quantized inside the GEMM to MXFP4
 * (E2M1 elements, one E8M0 scale per 32 consecutive K) and multiplied against a
 * weight W[N,K] that was quantized to MXFP4 and preshuffled once; the product is
 * accumulated in FP32 and written as BF16 C[M,N]. Scope (same page, Scope): gfx950
 * only, N divisible by 256, K divisible by 128 (this library also caps N at 2^30 and K
 * at 2^24); rows of C at or beyond M are never read or written (same page,
 * Implementation: M-tail masking).
 *
 * Quantization rule (all entry points): for each 32-element block along K, the scale
 * byte is s = max(E - 2, 0) where E is the exponent field of the block's largest
 * magnitude (equivalently e = floor(log2 amax) - 2 clamped to [-127, 127], s = e + 127;
 * an all-zero block gets 0); each element x becomes the E2M1 code nearest to
 * x * 2^-e, ties to the even code, magnitudes >= 6 saturating to 6, with the sign bit
 * of x kept (so -0.0 encodes as 0x8).
 *
 * Conventions shared by every entry point:
 *  - All buffer pointers are device pointers, caller-allocated and caller-owned, and
 *    16-byte aligned. The library allocates no device memory and keeps no per-call state.
 *  - Matrices are dense row-major. bf16 values are raw 16-bit patterns.
 *  - Argument errors are returned synchronously before any HIP call is made.
 *  - Work is enqueued on `stream` (NULL = the default stream); no entry point
 *    synchronizes the host. Faults inside a kernel surface at the caller's next sync.
 *  - Inputs must be finite; NaN/Inf inputs give unspecified (but in-bounds) results.
 *  - Output is bitwise reproducible for a given (M, N, K), device and library build.
 *  - Entry points are thread-safe.
 */
#ifndef MX_H_
#define MX_H_

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mx_status {
  MX_OK = 0,
  MX_ERR_NULL = 1,      /* a required pointer is NULL */
  MX_ERR_SHAPE = 2,     /* a size is negative or breaks a divisibility rule */
  MX_ERR_ALIGN = 3,     /* a pointer is not 16-byte aligned */
  MX_ERR_DEVICE = 4,    /* the current device is not gfx950 */
  MX_ERR_WORKSPACE = 5, /* a required workspace is missing or too small */
  MX_ERR_HIP = 6        /* a HIP runtime call or kernel launch failed */
} mx_status;

/* Static, human-readable name of a status code. Never NULL. */
const char* mx_status_string(mx_status s);

/* Version of the prepared-weight layout; a blob is only valid for the version that wrote it. */
int mx_prepared_layout_version(void);

/*
 * Size in bytes of a prepared MXFP4 weight of shape [N, K]: N*K/2 bytes of packed E2M1
 * payload followed by N*K/32 bytes of E8M0 scales, N*K*17/32 in all, e.g. 32,169,984
 * bytes for 8448 x 7168 ("[gfx950][FlyDSL] Add direct dense A4W4 MXFP4 GEMM", Model
 * validation). Returns 0 when N <= 0, K <= 0, N % 256, K % 128, N > 2^30 or K > 2^24.
 */
size_t mx_prepared_weight_bytes(int64_t N, int64_t K);

/*
 * One-time weight preparation ("prepare_gemm_a4w4_weight" of the page above,
 * Implementation: one-time packed E2M1 weight and E8M0 scale preshuffle).
 * w_bf16: [N, K] bf16 row-major (read only).
 * w_prep: mx_prepared_weight_bytes(N, K) bytes, written completely (opaque layout).
 * Requires N % 256 == 0, K % 128 == 0. Errors: MX_ERR_NULL, MX_ERR_SHAPE, MX_ERR_ALIGN,
 * MX_ERR_DEVICE, MX_ERR_HIP.
 */
mx_status mx_prepare_weight(const void* w_bf16, int64_t N, int64_t K, void* w_prep,
                            hipStream_t stream);

/*
 * Weight preparation from an already-quantized weight: the caller's packed E2M1 codes and
 * E8M0 scales are preshuffled once, as they are ("[gfx950][FlyDSL] Add direct dense A4W4
 * MXFP4 GEMM", Scope: packed E2M1 weights and E8M0 scales, preshuffled once).
 * w_fp4: [N, K/2] bytes, row n holding W[n, 2i] in the low nibble and W[n, 2i+1] in the
 * high nibble of byte i. w_scale: [N, K/32] bytes, the E8M0 scale of each 32-block along
 * K (value 2^(byte - 127)). Both read only. w_prep: mx_prepared_weight_bytes(N, K) bytes,
 * written completely. Every byte is copied as given; a scale byte of 255 (NaN in the OCP
 * MX encoding) is outside the contract. For a weight quantized by the rule above, the
 * result is identical to mx_prepare_weight's, and mx_unprepare_weight returns the inputs
 * unchanged. Same shape rules and errors as mx_prepare_weight.
 */
mx_status mx_prepare_weight_packed(const void* w_fp4, const void* w_scale, int64_t N, int64_t K,
                                   void* w_prep, hipStream_t stream);

/*
 * Test support: the inverse of the preshuffle. Writes the canonical MXFP4 form of a
 * prepared weight: w_fp4 [N, K/2] (element at even k in the low nibble) and
 * w_scale [N, K/32] (one E8M0 byte per 32-block). Same shape rules and errors as
 * mx_prepare_weight.
 */
mx_status mx_unprepare_weight(const void* w_prep, int64_t N, int64_t K, void* w_fp4,
                              void* w_scale, hipStream_t stream);

/*
 * Standalone activation quantizer: the same rule as the GEMM's inline quantization,
 * written out in canonical layout ("[gfx1250] Fuse A4W4 stage1 FP4 quantization",
 * Summary: the standalone quant path).
 * a_bf16: [M, K] bf16. a_fp4: [M, K/2] bytes (low nibble = even k). a_scale: [M, K/32]
 * bytes. Requires M >= 0, K > 0, K % 32 == 0. M == 0 is a no-op returning MX_OK.
 */
mx_status mx_quant_act(const void* a_bf16, int64_t M, int64_t K, void* a_fp4, void* a_scale,
                       hipStream_t stream);

/*
 * Workspace the dense GEMM can use at this shape: FP32 partial sums of a split-K
 * reduction (few rows), or, at large M, the activations quantized once into the
 * prepared layout (M rounded up to 64, times K * 17 / 32 bytes), followed, when the
 * 128 x 128 output tiles slightly exceed one round of the chip, by the FP32 partial tiles
 * of the tail tiles' K slices (from the next 256-byte boundary). It is always optional:
 * with a NULL or smaller workspace the library picks a configuration that needs less or
 * none; results stay within the same bound, and are bitwise equal where no K slices are
 * involved (K slices add their partial sums in slice order). 0 for an invalid shape.
 */
size_t mx_a4w4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * The dense A4W4 GEMM ("flydsl_gemm_a4w4" of "[gfx950][FlyDSL] Add direct dense A4W4
 * MXFP4 GEMM", Summary and Implementation): C = Q(A) * Q(W)^T with Q the MXFP4
 * quantization above; A is quantized inside the kernel, never written to memory, except
 * that at large M with a big enough workspace its MXFP4 codes are written once into the
 * workspace and read back by the product kernel (bit-identical results).
 * a_bf16: [M, K] bf16. w_prep: prepared weight of shape [N, K]. c_bf16: [M, N] bf16,
 * rows < M written with the FP32 sum rounded to nearest even. Requires 0 <= M <= 2^30,
 * N % 256 == 0, K % 128 == 0, N <= 2^30, K <= 2^24. M == 0 is a no-op. workspace may be
 * NULL (then workspace_bytes is ignored); a non-NULL workspace must be 16-byte aligned.
 * The call is asynchronous on stream; workspace must stay alive until it completes.
 */
mx_status mx_a4w4_gemm(const void* a_bf16, const void* w_prep, void* c_bf16, int64_t M,
                       int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                       hipStream_t stream);

/*
 * For callers that cannot allocate device memory (code under stream capture, tight serving
 * loops, harnesses that forbid allocation): mx_a4w4_gemm with the plan it runs when handed
 * mx_a4w4_gemm_workspace_bytes(M, N, K) of workspace, that workspace being the library's own
 * device array of mx_noalloc_scratch_bytes() bytes (32 MiB), one per GPU, held until the
 * process ends; the call allocates and frees nothing. Same arguments, shape rules and results
 * as mx_a4w4_gemm without the workspace pair. MX_ERR_WORKSPACE when the plan needs more than
 * the array holds (e.g. the quantize-once plan at M * K * 17 / 32 > 32 MiB); nothing is
 * launched then. Every call on a GPU shares that GPU's array: calls that overlap on one GPU
 * (concurrent streams, threads) race and must be serialized by the caller. Nothing in the
 * array needs clearing between calls (each plan writes what it reads).
 */
mx_status mx_a4w4_gemm_noalloc(const void* a_bf16, const void* w_prep, void* c_bf16, int64_t M,
                               int64_t N, int64_t K, hipStream_t stream);

/* Size in bytes of the scratch array mx_a4w4_gemm_noalloc uses. Host only. */
size_t mx_noalloc_scratch_bytes(void);

/*
 * A16WFP4 variant (named in "[gfx950][FlyDSL] Add direct dense A4W4 MXFP4 GEMM", CI Guide, as
 * outside that change): C[M, N] = A[M, K] x W^T with the bf16 activations NOT quantized and
 * W the prepared MXFP4 weight decoded to real values (E2M1 value x 2^(scale - 127), exact
 * in bf16; weight blocks with scale byte 0, block amax below 2^-125, may decode to zero);
 * FP32 accumulation on the bf16 MFMA, bf16 output (round to nearest even); rows >= M are
 * untouched. Same arguments, shape rules and errors as mx_a4w4_gemm, without a workspace.
 */
mx_status mx_a16w4_gemm(const void* a_bf16, const void* w_prep, void* c_bf16, int64_t M,
                        int64_t N, int64_t K, hipStream_t stream);

/*
 * Grouped MoE GEMM1 (expert-segmented dense GEMM, "[HIP] [CK] [FlyDSL] [Kernel] Extend
 * MXFP4 GEMM1 replacement to A4W4", Summary; shape of "[gfx1250] Fuse A4W4 stage1 FP4
 * quantization", Performance). Output row r (expert-sorted order) is
 * Q(A[row_token[r]]) * Q(W_e)^T for the expert e with
 * expert_offsets[e] <= r < expert_offsets[e+1].
 * a_bf16: [T, K] bf16. row_token: [R_max] int32 device array; entries below R are token
 * indices in [0, T) (an index outside that range reads as an all-zero row).
 * expert_offsets: [E+1] int32 device array, non-decreasing, expert_offsets[0] == 0,
 * expert_offsets[E] == R <= R_max (segments are clamped to [0, R_max]).
 * w_prep_stacked: E prepared weights of shape [N, K],
 * expert e at byte offset e * mx_prepared_weight_bytes(N, K) (64-bit addressing).
 * c_bf16: [R_max, N] bf16; rows >= R are untouched. rows_hint: the expected rows per
 * active expert (only a tiling hint; any value >= 1 is correct).
 * Requires E >= 1, T >= 0, R_max >= 0, N % 256 == 0, K % 128 == 0.
 */
mx_status mx_a4w4_gemm_grouped(const void* a_bf16, const int32_t* row_token,
                               const int32_t* expert_offsets, int64_t E, int64_t R_max,
                               const void* w_prep_stacked, void* c_bf16, int64_t T, int64_t N,
                               int64_t K, int64_t rows_hint, hipStream_t stream);

/*
 * Second MoE GEMM (the stage after GEMM1 in "[HIP] [CK] [FlyDSL] [Kernel] Extend MXFP4 GEMM1
 * replacement to A4W4", Summary) on activation rows that are already MXFP4: output row r
 * (expert-sorted order) is Q_r * Q(W_e)^T for the expert e with
 * expert_offsets[e] <= r < expert_offsets[e+1], where Q_r is MXFP4 row r given in
 * canonical form (a_fp4 [R_max, K/2] bytes, element at even k in the low nibble; a_scale
 * [R_max, K/32] E8M0 bytes, 255 outside the contract), e.g. the output of
 * mx_a4w4_gemm_grouped_act_quant or mx_quant_act. No quantization takes place; the sums
 * accumulate in FP32 and are written as bf16 to c_bf16 [R_max, N] (rows >= R untouched).
 * expert_offsets, w_prep_stacked and rows_hint as for mx_a4w4_gemm_grouped.
 * Requires E >= 1, R_max >= 0, N % 256 == 0, K % 128 == 0. Errors: MX_ERR_NULL,
 * MX_ERR_SHAPE, MX_ERR_ALIGN, MX_ERR_DEVICE, MX_ERR_HIP.
 */
mx_status mx_a4w4_gemm_grouped_mx(const void* a_fp4, const void* a_scale, const int32_t* expert_offsets,
                                  int64_t E, int64_t R_max, const void* w_prep_stacked, void* c_bf16,
                                  int64_t N, int64_t K, int64_t rows_hint, hipStream_t stream);

/*
 * Top-k weighted combine of per-row outputs into per-token outputs:
 * out[t, n] = sum over k < topk of token_weights[t, k] * y[token_rows[t, k], n], summed in
 * FP32 in k order and rounded once to bf16 (round to nearest even); a row index outside
 * [0, R) contributes nothing. y_bf16: [R, N] bf16 (e.g. the output of
 * mx_a4w4_gemm_grouped_mx). token_rows: [T, topk] int32; token_weights: [T, topk] float32;
 * out_bf16: [T, N] bf16. Requires R >= 0, T >= 0, 1 <= topk <= 1024, N > 0, N % 8 == 0.
 * T == 0 is a no-op. Errors: MX_ERR_NULL, MX_ERR_SHAPE, MX_ERR_ALIGN (y, out: 16 bytes;
 * token_rows, token_weights: 4 bytes), MX_ERR_DEVICE, MX_ERR_HIP.
 */
mx_status mx_moe_combine(const void* y_bf16, int64_t R, const int32_t* token_rows,
                         const float* token_weights, int64_t T, int64_t topk, int64_t N,
                         void* out_bf16, hipStream_t stream);

/* Activation of the fused GEMM1 epilogue. */
enum { MX_ACT_SILU = 0, MX_ACT_SWIGLU = 1 };

/*
 * Grouped MoE GEMM1 with the activation and the MXFP4 quantization for the second GEMM
 * fused into its epilogue ("[gfx1250] Fuse A4W4 stage1 FP4 quantization", Summary: the
 * GEMM1 epilogue emits packed MXFP4 payloads and E8M0 scales directly after SiLU or
 * SwiGLU, the scale computed from the FP32 activation value). Routing, segments and
 * weights are those of mx_a4w4_gemm_grouped; for output row r with GEMM1 row c (FP32):
 *   act == MX_ACT_SWIGLU: h[j] = SiLU(c[j]) * c[N/2 + j], j < Nh = N/2 (gate columns first);
 *   act == MX_ACT_SILU:   h[j] = SiLU(c[j]), j < Nh = N;  SiLU(x) = x / (1 + exp(-x)),
 * evaluated in FP32 with the hardware exponential and reciprocal (relative error at most
 * (|x| + 8) * 2^-23).
 * h is quantized along its columns with the rule at the top of this file applied to the
 * FP32 value of h (E8M0 scale from the FP32 block amax, one conversion to E2M1) and written
 * in canonical form: h_fp4 [R_max, Nh/2] bytes (element at even j in the low nibble),
 * h_scale [R_max, Nh/32] bytes; rows >= R are untouched. Because h is formed in FP32 from
 * FP32 accumulators, a code or scale whose exact value lies at a rounding boundary may
 * differ from the exact product's by one step. Requirements and errors as for
 * mx_a4w4_gemm_grouped, plus act in {MX_ACT_SILU, MX_ACT_SWIGLU} (else MX_ERR_SHAPE).
 */
mx_status mx_a4w4_gemm_grouped_act_quant(const void* a_bf16, const int32_t* row_token,
                                         const int32_t* expert_offsets, int64_t E, int64_t R_max,
                                         const void* w_prep_stacked, int64_t T, int64_t N, int64_t K,
                                         int32_t act, int64_t rows_hint, void* h_fp4, void* h_scale,
                                         hipStream_t stream);

/*
 * Introspection (host only, no GPU needed): the kernel instantiation(s) mx_a4w4_gemm
 * would launch for (M, N, K) with a workspace of workspace_bytes, e.g.
 * "k_gemm_tile<1, 4, 4, 4, 1, 2> GM=8" or "k_gemm_stream<1, 1, 2, 16, 1> S=1", written
 * NUL-terminated (truncated to buf_len) into the caller's host buffer; "none" for M == 0.
 * The names match the kernel names a profiler reports. Honours the library's tuning
 * override (environment variable MX_GEMM_CONFIG) like the GEMM itself. Errors:
 * MX_ERR_SHAPE (as mx_a4w4_gemm), MX_ERR_NULL (buf NULL or buf_len 0), MX_ERR_HIP (the
 * override names no configuration that can run this call; the GEMM would fail the same way).
 */
mx_status mx_a4w4_gemm_plan(int64_t M, int64_t N, int64_t K, size_t workspace_bytes, char* buf,
                            size_t buf_len);

/*
 * Introspection (host only, no GPU needed): the kernel instantiation mx_a16w4_gemm would
 * launch for (M, N, K): "k_gemm_a16w4_stream<MT, NG, WK, PD>" (decode M, at most 32 rows) or
 * "k_gemm_a16w4 (64 x 256 tiles)", written NUL-terminated (truncated to buf_len) into the
 * caller's host buffer; "none" for M == 0. Errors: MX_ERR_SHAPE (as mx_a16w4_gemm),
 * MX_ERR_NULL (buf NULL or buf_len 0).
 */
mx_status mx_a16w4_gemm_plan(int64_t M, int64_t N, int64_t K, char* buf, size_t buf_len);

/*
 * The same for mx_a4w4_gemm_grouped with E experts, R_max rows and T tokens (the choice
 * may depend on any of them; tuning override MX_GROUPED_CONFIG); "none" for R_max == 0. Same shape rules and errors as the grouped
 * GEMM, plus MX_ERR_NULL for buf.
 */
mx_status mx_a4w4_gemm_grouped_plan(int64_t E, int64_t R_max, int64_t T, int64_t N, int64_t K,
                                    int64_t rows_hint, char* buf, size_t buf_len);

/*
 * The same for mx_a4w4_gemm_grouped_act_quant (its kernel depends on E, R_max, N, act and
 * the hint, as for the call; tuning override MX_GROUPED_CONFIG="gt,..."). Errors:
 * MX_ERR_SHAPE (E, R_max, shape or act as for the call), MX_ERR_NULL (buf), MX_ERR_HIP (the
 * override names no fused configuration for N).
 */
mx_status mx_a4w4_gemm_grouped_act_quant_plan(int64_t E, int64_t R_max, int64_t N, int64_t K,
                                              int32_t act, int64_t rows_hint, char* buf,
                                              size_t buf_len);

/* The same for mx_a4w4_gemm_grouped_mx (its kernel depends on N, K and the hint). Errors as
 * for mx_a4w4_gemm_grouped_act_quant_plan. */
mx_status mx_a4w4_gemm_grouped_mx_plan(int64_t N, int64_t K, int64_t rows_hint, char* buf,
                                       size_t buf_len);

/* ------------------------------------------------------------------------------------------
 * Routing to experts, and the tables that the grouped GEMMs and the combine take: what stands
 * between a router's logits and mx_a4w4_gemm_grouped / mx_moe_combine.
 * ------------------------------------------------------------------------------------------ */

/* Score of an expert's logit, and the type of the logits. */
enum { MX_SCORE_SOFTMAX = 0, MX_SCORE_SIGMOID = 1 };
enum { MX_TYPE_BF16 = 0, MX_TYPE_F32 = 1 };

/*
 * The topk experts of each token and their weights. With l = logits[t]:
 *   s[e] = softmax(l)[e] or 1 / (1 + exp(-l[e]));   c[e] = s[e] + bias[e]  (s[e] where bias is NULL);
 *   groups > 1: the experts stand in `groups` groups of E / groups neighbours; a group's value is the
 *     sum of its group_top (1 or 2) largest c, and only the topk_groups best groups stay;
 *   topk_ids[t]: the topk experts with the largest c of those, largest first;
 *   topk_weights[t][i] = scale * s[id], with renormalize != 0 over the sum of s over the chosen (0
 *     where that sum is 0).
 * Equal c go to the lower expert, equal values to the lower group. c and values are FP64 and are
 * compared to 42 bits, to which c is cut and a value, the sum of c as they are, rounded (without a
 * bias c is compared by the logits, exactly); weights are formed in FP64 and rounded once. An expert
 * whose logit or bias is -inf or NaN is never chosen and has no part in any sum; a logit of +inf counts
 * as its type's largest number, a bias of +inf as float32's. Where fewer than topk experts are left, the
 * rest of the places get id -1 and weight 0; mx_moe_sort gives those no row.
 *  logits: row t's E values of logits_type at element t * logits_stride (any address of that type).
 *  bias: [E] float32, or NULL. num_rows: [1] int32 or NULL: rows from *num_rows on are padding, all
 *  of their places get id -1 and weight 0. topk_ids: [T, topk] int32, topk_weights: [T, topk] float32.
 * Requires 0 <= T <= 2^30 / topk, 1 <= E <= 1024, 1 <= topk <= min(64, topk_groups * E / groups),
 * 1 <= groups <= 64, E % groups == 0, 1 <= topk_groups <= groups, 0 <= logits_stride < 2^32, a finite
 * scale. T == 0 is a no-op. Errors: MX_ERR_NULL, MX_ERR_SHAPE, MX_ERR_ALIGN (logits: their type's
 * size; the others 4 bytes), MX_ERR_DEVICE, MX_ERR_HIP.
 */
mx_status mx_moe_route(const void* logits, int64_t logits_stride, int32_t logits_type, const float* bias,
                       int64_t T, int64_t E, int64_t topk, int32_t score, int64_t groups, int64_t topk_groups,
                       int32_t group_top, int32_t renormalize, float scale, const int32_t* num_rows,
                       int32_t* topk_ids, float* topk_weights, hipStream_t stream);

/*
 * The chosen experts sorted: the tables of mx_a4w4_gemm_grouped and mx_moe_combine for the E experts
 * first_expert .. first_expert + E - 1 (all of them, or one device's share). The places of topk_ids
 * [T, topk] whose id is among these are ordered by expert, those of one expert by token and place;
 * R is their number.
 *  expert_offsets: [E + 1] int32, where each expert's rows start; expert_offsets[E] = R.
 *  row_token: [T * topk] int32, the token of each row; -1 from row R on.
 *  token_rows: [T, topk] int32, the row of each place; -1 where the id is none of these experts'.
 * workspace: mx_moe_sort_workspace_bytes(T, topk, E) bytes (0 for few places: NULL), 16-byte aligned.
 * Requires T >= 0, 1 <= topk <= 1024, T * topk <= 2^28, 1 <= E <= 1024, 0 <= first_expert < 2^30. The
 * outputs may not overlap topk_ids. Errors: MX_ERR_NULL, MX_ERR_SHAPE, MX_ERR_ALIGN (4 bytes;
 * workspace 16), MX_ERR_WORKSPACE, MX_ERR_DEVICE, MX_ERR_HIP.
 */
mx_status mx_moe_sort(const int32_t* topk_ids, int64_t T, int64_t topk, int64_t first_expert, int64_t E,
                      int32_t* expert_offsets, int32_t* row_token, int32_t* token_rows, void* workspace,
                      size_t workspace_bytes, hipStream_t stream);

/* Workspace mx_moe_sort needs. 0 for sizes it refuses. */
size_t mx_moe_sort_workspace_bytes(int64_t T, int64_t topk, int64_t E);

/* ------------------------------------------------------------------------------------------
 * A key/value cache in MXFP4, in pages, and the attention that reads it: what a decoder
 * layer runs between the GEMM that makes its queries, keys and values and the one that takes
 * the attention's output. Keys and values are quantized row by row with the rule at the top
 * of this file (blocks of 32 along the head), so a cached head costs D * 17/32 bytes per key
 * and per value instead of 2 D.
 *
 * Cache layout. A cache is num_pages pages of page_size tokens (a power of two, 16 .. 1024)
 * for `heads` key/value heads of D elements (64, 128 or 256): [page][head] blocks of
 * page_size * D * 17 / 16 bytes. One block holds, with n = page_size / 16 tiles of 16 tokens
 * and m = D / 32 scale blocks per token,
 *   K codes   [n][m][16 tokens][16 bytes]    one 32-block each, canonical order
 *   V codes   [n][4][16 bytes][m][4 tokens]  byte b of block j of token 4g + i at [g][b][j][i]
 *   K scales  [n][m][16 tokens]              E8M0
 *   V scales  [n][16 tokens][m]              E8M0
 * (every region is an MFMA operand in lane order). Slot s is token s % page_size of page
 * s / page_size. A cache needs no clearing: bytes of tokens that were never written do not
 * reach any result. The rows given to mx_kv_write must be finite.
 * ------------------------------------------------------------------------------------------ */

/* Size in bytes of a cache. 0 when num_pages is not in [1, 2^31), heads not in [1, 1024], or
 * page_size or D is not one of those above. */
size_t mx_kv_cache_bytes(int64_t num_pages, int64_t page_size, int64_t heads, int64_t D);

/*
 * Block tables and slot maps from the requests' lengths, on the device (no host round trip,
 * fit for stream capture). Request b holds old_lens[b] tokens and shall hold new_lens[b]: it
 * takes ceil(new / page_size) - ceil(old / page_size) pages from the stack of free pages, or
 * gives its last pages back when that is negative (an ended request: new_lens[b] = 0; drafts
 * taken back: fewer than old).
 *  old_lens, new_lens: [B] int32. block_table: [B, max_blocks] int32, updated in place: entry
 *    [b][i] is the page of tokens i * page_size ..; only the entries of new pages are written.
 *  free_pages: [capacity] int32, the stack, updated in place; free_count: [1] int32, its
 *    height; free_count_out: [1] int32, the height afterwards (may be free_count itself).
 *    Pages given back are pushed first, in the requests' order and each request's in order of
 *    its tokens; then pages are popped in the requests' order.
 *  cu_q: [B+1] int32, where each request's new rows start: the sums of max(new - old, 0).
 *  slots: [T_max] int64 and positions: [T_max] int32, the slot and the position of every new
 *    row; both are -1 from row cu_q[B] on (so a padded batch writes nothing).
 *  status: [1] int32: 0; or the number of pages the stack lacks; or -1 when a length is
 *    negative or past max_blocks * page_size, the new rows exceed T_max, free_count is not in
 *    [0, capacity], or the pages given back do not fit the stack. Unless it is 0, nothing
 *    moves: the table and the stack keep their contents, free_count_out is free_count, cu_q
 *    is all 0 and every slot is -1.
 * Because the lengths and the height are read from one place and written to another, calling
 * it twice with the same arguments gives the same result. A page must stand on the stack or
 * in the table's held entries once. workspace: mx_kv_tables_workspace_bytes(B, T_max) bytes
 * (0 for small batches: NULL), 16-byte aligned. Requires 0 <= B <= 2^20, 1 <= max_blocks,
 * max_blocks * page_size <= 2^30, 0 <= T_max <= 2^30, 0 <= capacity < 2^31 and page_size as above. Errors: MX_ERR_NULL,
 * MX_ERR_SHAPE, MX_ERR_ALIGN (4 bytes; slots 8; workspace 16), MX_ERR_WORKSPACE,
 * MX_ERR_DEVICE, MX_ERR_HIP.
 */
mx_status mx_kv_tables(const int32_t* old_lens, const int32_t* new_lens, int64_t B, int64_t page_size,
                       int32_t* block_table, int64_t max_blocks, int32_t* free_pages, int64_t capacity,
                       const int32_t* free_count, int32_t* free_count_out, int64_t T_max, int32_t* cu_q,
                       int64_t* slots, int32_t* positions, int32_t* status, void* workspace,
                       size_t workspace_bytes, hipStream_t stream);

/* Workspace mx_kv_tables needs. 0 for sizes it refuses. */
size_t mx_kv_tables_workspace_bytes(int64_t B, int64_t T_max);

/*
 * Quantizes T rows of keys and of values into the cache: row t's head h goes to slot
 * slots[t]. k_bf16, v_bf16: row t's heads are heads * D consecutive bf16 values at element
 * t * k_stride (t * v_stride), so columns of a fused projection's output can be given as they
 * are; strides are multiples of 8. slots: [T] int64; a slot outside [0, num_pages *
 * page_size) writes nothing. A slot named twice ends up with bytes of either row: give each
 * once. T == 0 is a no-op. Errors: MX_ERR_NULL, MX_ERR_SHAPE, MX_ERR_ALIGN (k, v, cache: 16
 * bytes; slots: 8), MX_ERR_DEVICE, MX_ERR_HIP.
 */
mx_status mx_kv_write(const void* k_bf16, int64_t k_stride, const void* v_bf16, int64_t v_stride,
                      const int64_t* slots, int64_t T, void* cache, int64_t num_pages, int64_t page_size,
                      int64_t heads, int64_t D, hipStream_t stream);

/*
 * The inverse: the values that the cache holds at `slots`, in bf16 (exact; a value below
 * bf16's least subnormal becomes 0 or that): k_bf16, v_bf16 [T, heads, D] dense. Rows whose
 * slot is outside the cache are left as they were. Same requirements and errors.
 */
mx_status mx_kv_read(const void* cache, int64_t num_pages, int64_t page_size, int64_t heads, int64_t D,
                     const int64_t* slots, int64_t T, void* k_bf16, void* v_bf16, hipStream_t stream);

/*
 * Attention of bf16 queries over the cache. Request b's rows are cu_q[b] .. cu_q[b+1] - 1 of
 * q; with n of them and L = kv_lens[b] cached tokens, row i stands at position L - n + i (its
 * own key is already in the cache) and
 *   out[i][h] = sum_j p_j V[j][h / (heads_q / heads)],  p = softmax_j(scale * q[i][h] . K[j])
 * over the tokens j < L that it sees: with causal != 0 those at j <= its position, and with
 * window > 0 (causal only) those at j > its position - window. A row that sees nothing is 0.
 *  q_bf16: row t's heads_q * D values at element t * q_stride; out_bf16 likewise with
 *    out_stride >= heads_q * D (strides are multiples of 8). heads_q is a multiple of heads.
 *    Rows from cu_q[B] on are neither read nor written.
 *  block_table: [B, max_blocks] int32; entries of tokens that no row sees are not read. An
 *    entry outside [0, num_pages) makes its tokens unseen.
 *  cu_q: [B+1] int32, non-decreasing from 0 (clamped to [0, T]); kv_lens: [B] int32 (clamped
 *    to [0, max_blocks * page_size]).
 *  max_q, max_kv: the most rows and the longest kv_len of any request: hints that choose the
 *    kernels, their cuts and the workspace, right at any value >= 1.
 *  workspace: partial results where the tokens of a request are split over the chip, of
 *    mx_kv_attention_workspace_bytes(...) bytes; always optional: with a NULL or smaller one
 *    the tokens are split less or not at all. Calls that may overlap need one each; nothing in
 *    it needs clearing.
 * Queries are not quantized: elements down to 2^-13 of their row's largest are used exactly,
 * smaller ones to within 2^-21 of it. Scores and the softmax's maximum and sum are FP32; the
 * weights are rounded to bf16 for the product with V, whose sum is FP32; the result is rounded
 * once. Output is bitwise reproducible for the same arguments; which kernels run, and so the last
 * bits, go by all sizes and hints. A head of a row whose elements are not all finite is unspecified
 * itself and changes no other.
 * The sums have to stay in FP32's range, for each row over the tokens it sees: the sum over d of
 * |q_d K_d|, and scale times it, below 1e38; each element's sum of |V| over the tokens below
 * 2^120 (the weights reach 2^8 before the division).
 * Requires 0 <= T <= 2^30 / heads_q, heads_q <= 1024, 0 <= B <= 2^22 / heads (and 2^20),
 * 1 <= max_blocks, max_blocks * page_size <= 2^30, 0 < scale <= 2^127 and the cache's sizes as
 * above. T == 0 or B == 0 is a no-op. Errors: MX_ERR_NULL, MX_ERR_SHAPE,
 * MX_ERR_ALIGN (q, out, cache, workspace: 16 bytes; tables: 4), MX_ERR_DEVICE, MX_ERR_HIP.
 */
mx_status mx_kv_attention(const void* q_bf16, int64_t q_stride, const void* cache, int64_t num_pages,
                          int64_t page_size, const int32_t* block_table, int64_t max_blocks,
                          const int32_t* cu_q, const int32_t* kv_lens, int64_t B, int64_t T, int64_t heads_q,
                          int64_t heads, int64_t D, int64_t max_q, int64_t max_kv, int32_t causal,
                          int64_t window, float scale, void* out_bf16, int64_t out_stride, void* workspace,
                          size_t workspace_bytes, hipStream_t stream);

/* Workspace mx_kv_attention can use for these sizes. 0 where it needs none or refuses them. */
size_t mx_kv_attention_workspace_bytes(int64_t B, int64_t T, int64_t heads_q, int64_t heads, int64_t D,
                                       int64_t max_q, int64_t max_kv, int64_t window);

/*
 * Introspection (host only, no GPU needed): the kernels mx_kv_attention would launch for these
 * sizes with workspace_bytes of workspace, as the other *_plan calls. Errors: MX_ERR_SHAPE,
 * MX_ERR_NULL (buf NULL or buf_len 0).
 */
mx_status mx_kv_attention_plan(int64_t B, int64_t T, int64_t heads_q, int64_t heads, int64_t D, int64_t max_q,
                               int64_t max_kv, int64_t window, size_t workspace_bytes, char* buf,
                               size_t buf_len);

/* How mx_kv_append pairs the elements that it rotates: i with i + rot / 2, or 2 i with 2 i + 1. */
enum { MX_ROPE_HALVES = 0, MX_ROPE_PAIRS = 1 };

/*
 * What stands between the projection to queries, keys and values and mx_kv_attention, in one pass:
 * norms of each head, rotation by position, and the keys and values into the cache. For every head x
 * [D] of row t's queries and keys:
 *   y = x * weight / sqrt(max(mean(x^2) + eps, 2^-126))      (y = x where weight is NULL);
 *   element pairs (a, b) of the first `rot` elements, number i of rot / 2 of them, become
 *   (a cos - b sin, a sin + b cos) with the angle positions[t] * inv_freq[i], formed in FP64, and cos
 *   and sin times rope_scale.
 * Queries are worked out in FP32 (angles, and heads and weights past its range, in FP64) and rounded
 * once to bf16, to q_out. Keys are quantized as FP64 arithmetic, rounded to FP32, has them, values as they are,
 * both with the rule at the top of this file into slot slots[t] of the cache, as mx_kv_write does.
 *  q_bf16, k_bf16, v_bf16: row t's heads_q * D (heads * D) values at element t * q_stride (k_stride,
 *    v_stride); q_out likewise with q_out_stride >= heads_q * D. Strides are multiples of 8. q_out may
 *    be q_bf16 itself (with the same stride) and must not overlap any input otherwise.
 *  Without queries, q_bf16 NULL and heads_q 0; without keys and values (a layer that reads another's
 *    cache), k_bf16, v_bf16, slots and cache NULL, heads and num_pages 0.
 *  positions: [T] int32; a row whose position is below 0 is padding: nothing of it is written or
 *    reaches a result.
 *  slots: [T] int64; a slot outside [0, num_pages * page_size) writes no key and value (its queries
 *    are still done). Give each slot once.
 *  q_weight, k_weight: [D] float32 or NULL. inv_freq: [rot / 2] float32; NULL with rot 0 for none.
 * Requires 0 <= T <= 2^30, heads and heads_q at most 1024, one of them above 0, D 64, 128 or 256,
 * rot a multiple of 16 in [0, D], eps >= 0 and finite, a finite rope_scale, page_size as above (also
 * without keys). Elements, weights, frequencies and weights times rope_scale must be finite in FP32, and
 * so must keys after norm and rotation and, where q_weight is NULL, each a cos and b sin of the queries
 * (times rope_scale); angles must stay below 2^31. T == 0 is a no-op. Errors: MX_ERR_NULL, MX_ERR_SHAPE,
 * MX_ERR_ALIGN (q, k, v, q_out, cache: 16 bytes; slots: 8; the others 4), MX_ERR_DEVICE, MX_ERR_HIP.
 */
mx_status mx_kv_append(const void* q_bf16, int64_t q_stride, const void* k_bf16, int64_t k_stride,
                       const void* v_bf16, int64_t v_stride, const int32_t* positions, const int64_t* slots,
                       int64_t T, int64_t heads_q, int64_t heads, int64_t D, void* cache, int64_t num_pages,
                       int64_t page_size, const float* q_weight, const float* k_weight, float eps,
                       const float* inv_freq, int64_t rot, int32_t rope, float rope_scale, void* q_out,
                       int64_t q_out_stride, hipStream_t stream);

/*
 * Verification of drafted tokens against the target model's probabilities, and the next token, from
 * random numbers that the caller gives; the lengths it returns are mx_kv_tables' new_lens for the
 * following step (drafts taken back). Request b's rows are cu_q[b] .. cu_q[b+1] - 1, as for
 * mx_kv_attention: first its last token, then its drafts, so that tokens[r + 1] is what row r's
 * distribution p = target_probs[r] judges. From its first row on, with q = draft_probs[r], the draft
 * x = tokens[r + 1] is accepted while
 *   accept_random[r] * q[x] < p[x]     (q[x] = 1 where draft_probs is NULL: drafts without chance)
 * and, at the first row that refuses, the next token is drawn from max(p - q, 0) (p without x where
 * draft_probs is NULL; p itself where that is 0 everywhere); after the last draft it is drawn from p.
 * Drawn from w: the least j with w[0] + .. + w[j] > u * (sum of w), u = sample_random[b] in [0, 1). All
 * of this is FP64. Probabilities below 0 and NaN count as 0, +inf may not be given, and rows need not
 * sum to 1; u below 0 or NaN counts as 0 and above 1 as 1 (the last token with a weight); an
 * accept_random that is NaN and a draft outside [0, V) refuse.
 *  target_probs, draft_probs: row r's V float32 at element r * target_stride (r * draft_stride).
 *  tokens: [T] int32. cu_q: [B + 1] int32, non-decreasing from 0 (clamped to [0, T]). kv_lens: [B]
 *    int32, with this step's rows. accept_random: [T], sample_random: [B] float32.
 *  out_tokens: [T] int32: at a request's rows its accepted drafts, then the drawn token (-1 where p is
 *    0 everywhere), then -1; -1 from row cu_q[B] on.
 *  accepted: [B] int32, how many drafts. new_lens: [B] int32, kv_lens[b] less the refused drafts (kv_lens
 *    itself may be given; no other output may overlap an input).
 *  A request without rows has 0 accepted and keeps its length.
 * workspace: mx_verify_drafts_workspace_bytes(B, V) bytes, 16-byte aligned. Requires 0 <= T <= 2^30,
 * 0 <= B <= 2^16 - 2, 1 <= V <= 2^24, strides in [V, 2^32) (or 0). Errors: MX_ERR_NULL, MX_ERR_SHAPE,
 * MX_ERR_ALIGN (4 bytes; workspace 16), MX_ERR_WORKSPACE, MX_ERR_DEVICE, MX_ERR_HIP.
 */
mx_status mx_verify_drafts(const float* target_probs, int64_t target_stride, const float* draft_probs,
                           int64_t draft_stride, const int32_t* tokens, const int32_t* cu_q,
                           const int32_t* kv_lens, const float* accept_random, const float* sample_random,
                           int64_t T, int64_t B, int64_t V, int32_t* out_tokens, int32_t* accepted,
                           int32_t* new_lens, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Workspace mx_verify_drafts needs. 0 for sizes it refuses, and for B == 0. */
size_t mx_verify_drafts_workspace_bytes(int64_t B, int64_t V);

#ifdef __cplusplus
}
#endif

#endif /* MX_H_ */
