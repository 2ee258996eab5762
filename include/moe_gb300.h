/*
 * moe_gb300.h -- C ABI of the Mixture-of-Experts expert-layer hot path on GB300 (sm_103a).
 *
 * The path: top-k routing -> token-to-expert alignment (moe_align) -> geometric
 * token-dimension bucketing and padding (moe_bucket_pad) -> grouped GEMM1 + bias + SwiGLU
 * (or relu^2) -> grouped GEMM2 + bias * routing weight -> top-k combine (moe_forward; in
 * MXFP8 with h quantised between the GEMMs, moe_mx_quantize); a single grouped GEMM over
 * given operands (moe_grouped_gemm); a per-token-scaled FP8 grouped GEMM over per-expert
 * group sizes (moe_gemm_per_token); and the per-expert weight gradient (moe_wgrad).  Around
 * that path, for training: the router's auxiliary losses with their gradient
 * (moe_router_loss) and the expert activation with an MXFP8 checkpoint and its backward pass
 * (moe_act_checkpoint, moe_act_backward); and, for the dense layers beside the experts (a
 * shared expert, the router's projection), a matrix product with bias, activation and residual
 * in its epilogue and its backward products (moe_dense_gemm, moe_dense_bias_grad), and the sum
 * of a token's pair rows (moe_pair_sum).  Between layers: dropout, the residual's addition and the
 * RMS norm, whose output can be the 8-bit operands of the calls above (moe_residual_norm,
 * moe_residual_norm_backward); beside a dense layer: the low-rank adapters of many requests
 * (moe_adapter_gemm).
 *
 * Sources of the definitions (pull-request pages):
 *  [BUCKET] "Bound Triton MoE JIT specializations via token-dim bucketing and warmup",
 *           TensorRT-LLM PR 15311 -- Description; Test Coverage.
 *  [DECODE] "tune the Nemotron MTP decode row on S5000 with a checked-in recipe",
 *           torchada PR 115 -- What it does (tiny-M bf16 fused-MoE decode shape).
 *  [AITER]  "Add MoE GEMM variants and weight-gradient kernel", ROCm aiter PR 5310 --
 *           Summary; Notes; second review (sentinel handling, E8M0 decoding, bias indexing).
 *
 * Conventions for every call
 *  - All device buffers are owned by the caller.  The library never allocates device
 *    memory; scratch comes from ctx->workspace (size from the *_workspace_size calls).
 *  - Work is enqueued on ctx->stream (a cudaStream_t; NULL = the legacy default stream).
 *    No call synchronises the host with the device.
 *  - Every device pointer must be 16-byte aligned and every tensor dense row-major with
 *    exactly the shape stated (a per-expert bias is a contiguous [E, N] array; strided
 *    biases are not accepted -- the bias-stride defect named in [AITER]'s second review
 *    is ruled out by contract).
 *  - Integers that index pairs or weight elements are 64-bit inside the kernels: with
 *    E = 256 an expert offset times the per-expert weight size exceeds INT32_MAX ([AITER],
 *    Notes).
 *  - The return value reports argument and launch errors only.  Errors that depend on
 *    the data (an expert id outside [0, E), an activation outside the decode path's
 *    float16 range) are written to the optional device word ctx->dev_status, first error
 *    wins; the caller reads it after synchronising.  No kernel traps.
 *  - moe_last_error() returns a thread-local description of the last failed call.
 *  - The library keeps no state; calls are thread-safe.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t moe_status;
#define MOE_OK 0
#define MOE_WARN_PAD_IGNORED 1    /* moe_bucket_pad: padding not allowed for this mode   */
#define MOE_ERR_INVALID_ARG (-1)  /* null pointer, bad size, misalignment               */
#define MOE_ERR_UNSUPPORTED (-2)  /* a size or mode this build does not implement       */
#define MOE_ERR_CAPACITY (-3)     /* an output or workspace buffer is too small         */
#define MOE_ERR_CUDA (-4)         /* a CUDA launch or runtime error                     */
/* device status codes (ctx->dev_status) */
#define MOE_ERR_INVALID_EXPERT (-5) /* a top-k id outside [0, E)                        */
#define MOE_ERR_RANGE (-6)          /* an activation or h value beyond float16's 65504   */
#define MOE_ERR_TIMEOUT (-7)        /* a bounded wait inside a kernel ran out            */

typedef enum {
  MOE_Q_BF16 = 0,        /* bf16 weights, bf16 activations                              */
  MOE_Q_MXFP4_W4A16 = 1, /* E2M1 weights, two per byte (even K index in the low nibble),
                            one E8M0 scale per 32 along K; bf16 activations            */
  MOE_Q_MXFP8 = 2        /* E4M3 weights and activations, one E8M0 scale per 32 along K */
} moe_quant;

typedef struct {
  void* stream;            /* cudaStream_t                                                  */
  void* workspace;         /* device scratch, caller-owned, 256-byte aligned                */
  size_t workspace_bytes;  /* its size                                                      */
  int32_t* dev_status;     /* optional device int32 (set to 0 by the caller); may be NULL   */
  void** events;           /* optional host array of cudaEvent_t recorded on the stream
                              around each kernel of a call (profiling); may be NULL.
                              moe_forward: [0] before GEMM1 (after x's f16 copy or
                              planes), [1] after GEMM1, [2] after GEMM2, [3] after the
                              combine (needs n_events >= 4);
                              moe_grouped_gemm, moe_wgrad: [0] before, [1] after.      */
  int32_t n_events;
} moe_ctx;

/* Thread-local text of the last error returned on this thread ("" if none). */
const char* moe_last_error(void);

/* ------------------------------------------------------------------------------------ *
 * Alignment: routing + moe_align_block_size                                             *
 * ------------------------------------------------------------------------------------ */

/* Capacity of the alignment outputs for num_pairs = T*k pairs:
 *   cap_tokens = round_up(num_pairs + E*(block_m-1), block_m), cap_blocks = cap_tokens/block_m
 * -- the most slots any routing can need (each expert's count padded up to whole
 * blocks). */
moe_status moe_align_capacity(int64_t num_pairs, int32_t E, int32_t block_m,
                              int64_t* cap_tokens, int64_t* cap_blocks);

/* Routing and alignment (one call).
 *
 * Routing (when logits != NULL): logits [T, E] fp32 -> topk_ids [T, k] int32 (the k largest
 * logits in descending order; equal logits rank the lower expert id first) and topk_w
 * [T, k] fp32 = softmax over the k chosen logits, computed in float64 and rounded to
 * float32.  When logits == NULL, topk_ids is an input and topk_w is not touched (may be
 * NULL).
 *
 * Alignment ([AITER] Summary and second review; [DECODE] What it does): with pair index
 * p = t*k + j, c_e pairs routed to expert e, P_e = c_e rounded up to block_m and
 * O_e = sum_{e'<e} P_e':
 *   sorted_token_ids[cap_tokens]: slots O_e .. O_e+c_e-1 hold expert e's pair indices in
 *       ascending order; every other slot holds the sentinel T*k;
 *   expert_ids[cap_tokens/block_m]: block b holds the expert owning slots
 *       b*block_m .. (b+1)*block_m-1, and -1 for every block at or past
 *       num_tokens_post_padded/block_m (kernels skip -1 blocks at once);
 *   num_tokens_post_padded[1] = sum_e P_e;
 *   expert_offsets[E+1] (may be NULL) = unpadded prefix sums of c_e (differences are the
 *       per-expert group sizes).
 * Limits: 1 <= k <= 32, k <= E <= 1024, 1 <= block_m <= 1024, 0 <= T, T*k < 2^31.
 * cap_tokens must be >= moe_align_capacity() and a multiple of block_m
 * (MOE_ERR_CAPACITY).  Out-of-range ids set MOE_ERR_INVALID_EXPERT in dev_status and are
 * left out of the outputs.  Needs no workspace. */
moe_status moe_align(const float* logits, int32_t* topk_ids, float* topk_w,
                     int64_t T, int32_t k, int32_t E, int32_t block_m,
                     int32_t* sorted_token_ids, int64_t cap_tokens,
                     int32_t* expert_ids, int32_t* num_tokens_post_padded,
                     int32_t* expert_offsets, const moe_ctx* ctx);

/* ------------------------------------------------------------------------------------ *
 * Token-dimension bucketing ([BUCKET] Description, Test Coverage)                        *
 * ------------------------------------------------------------------------------------ */

/* bucket(m) = ceil(m / s) * s with s = max(1, 2^(floor(log2 m) - 3)): eight buckets per
 * power-of-two octave from 16 on, every m < 16 its own bucket, at most 12.5% padding.
 * Returns -1 for m < 1. */
int64_t moe_bucket(int64_t m);

/* Number of buckets <= max_tokens (97 for 20000). */
int64_t moe_bucket_count(int64_t max_tokens);

/* T_pad = bucket(T) for MOE_Q_MXFP4_W4A16; for every other mode padding is not allowed
 * (dynamic activation scales would let pad rows change real outputs), *T_pad = T and the
 * call returns MOE_WARN_PAD_IGNORED.  T == 0 gives T_pad = 0.
 * Device part (optional): when x_pad != NULL, rows [0, T) of x ([T, row_bytes]) are copied
 * to x_pad ([T_pad, row_bytes]; x == x_pad skips the copy) and rows [T, T_pad) are zeroed;
 * likewise logits [T, E] fp32 -> logits_pad [T_pad, E] when logits_pad != NULL (zero pad
 * logits route pad rows to experts 0..k-1 with weight 1/k).  row_bytes must be a multiple
 * of 16. */
moe_status moe_bucket_pad(int64_t T, moe_quant quant, int64_t* T_pad,
                          const void* x, void* x_pad, int64_t row_bytes,
                          const float* logits, float* logits_pad, int32_t E,
                          const moe_ctx* ctx);

/* ------------------------------------------------------------------------------------ *
 * Forward: grouped GEMM1 + SwiGLU -> grouped GEMM2 -> combine                           *
 * ------------------------------------------------------------------------------------ */

/* Activation between the GEMMs.  MOE_ACT_RELU2 is the non-gated relu2_no_mul of [DECODE]
 * (the Nemotron recipe in its table of added files: GEMM1 N = 1856 = I, no gate product). */
typedef enum {
  MOE_ACT_SWIGLU = 0,     /* h = silu(gate) * up; GEMM1 has 2I rows (gate | up)           */
  MOE_ACT_RELU2 = 1,      /* h = max(a, 0)^2;     GEMM1 has I rows                        */
  MOE_ACT_NONE = 2        /* moe_dense_gemm only: no activation                           */
} moe_activation;

/* N1 = 2I for MOE_ACT_SWIGLU, I for MOE_ACT_RELU2. */
typedef struct {
  moe_quant quant;
  int32_t E, K, I;        /* experts, hidden size, intermediate size                      */
  const void* w1;         /* [E, N1, K] (MXFP4: [E, N1, K/2] bytes); SwiGLU: rows 0..I-1
                             gate, rows I..2I-1 up                                        */
  const uint8_t* w1_scale;/* [E, N1, K/32] E8M0 (NULL for bf16)                           */
  const void* b1;         /* [E, N1] bf16 or NULL                                         */
  const void* w2;         /* [E, K, I] (MXFP4: [E, K, I/2] bytes)                         */
  const uint8_t* w2_scale;/* [E, K, I/32] E8M0 (NULL for bf16)                            */
  const void* b2;         /* [E, K] bf16 or NULL                                          */
  int32_t activation;     /* moe_activation (a zero-initialised struct is SwiGLU)         */
} moe_weights;

/* Workspace bytes moe_forward needs for T_rows rows of top-k with an alignment of
 * cap_tokens slots (moe_align_capacity): h [rows_h, I] (f16 for MXFP4 weights, bf16 for bf16
 * weights), o [T_rows*k, K] fp32 and x as f16 [rows_x, K], each 256-byte aligned.  rows_h =
 * T_rows*k and rows_x = T_rows up to 256 rows; above that h and x may be kept in
 * alignment-slot order and rows_h = rows_x = cap_tokens, and two small regions (one bit per
 * output tile of each GEMM) follow, which mark tiles whose weight scales need the exact
 * second pass.  Up to 256 rows five more regions follow, for the block-scaled MXFP4 kernels:
 * x as eight E2M1 digit planes [T_rows, 8, kq(K)] bytes (two codes a byte) and their E8M0
 * scales [T_rows, sb(K)], h as eight planes [T_rows*k, 8, kq(I)] and scales [T_rows*k,
 * sb(I)], and a unit list [T_rows*k + 1, 16 bytes], where kq(n) = 64 * ceil(n / 128) and
 * sb(n) = 16 * ceil(ceil(n / 128) / 4).  Returns 0 for a negative argument. */
size_t moe_forward_workspace_size(int64_t T_rows, int32_t k, int32_t K, int32_t I, int64_t cap_tokens);

/* One MoE expert layer over the alignment of moe_align: both grouped GEMMs run as single
 * launches over every expert, each with an optional contiguous per-expert bias ([AITER]
 * Summary: the grouped GEMM over all experts in one launch with per-expert bias), and
 * token-dimension pad rows are computed like any other row but sliced off before the
 * top-k reduction, so only rows t < T_real reach y ([BUCKET] Description: padded rows are
 * removed ahead of the combine).  Blocks whose expert id is the -1 sentinel are skipped
 * before any weight is read ([AITER] second review: return at once on the sentinel).
 *
 * For every real token t < T_real (the others, e.g. bucket pad rows, are computed and
 * then sliced off):
 * Exactness of the W4A16 tensor-core path (above 256 rows): weights are decoded to float16
 * as code * 2^(E8M0 - 127), exact while that exponent lies in -23..13; a tile with a
 * nonzero block outside that window is computed again by a second pass with each weight row
 * shifted by a power of two (undone on its fp32 accumulator), so any E8M0 scale gives the
 * exact products the weight-streaming path gives below 256 rows.  Only a weight row whose
 * nonzero blocks span more than 36 octaves of scale is reported (MOE_ERR_RANGE).
 *
 *   gu = x_t . W1[e]^T + b1[e];  h = silu(gu[:I]) * gu[I:]  (SwiGLU) or
 *        h = max(gu, 0)^2  (relu^2; a NaN stays NaN)  (fp32, then rounded to the operand
 *        type of GEMM2: f16 RNE for MXFP4 weights -- |h| > 65504 sets MOE_ERR_RANGE, and so
 *        does |x| > 65504 where x is converted to f16: above 256 rows and for relu^2 -- and
 *        bf16 RNE for bf16 weights).  Up to 256 rows the MXFP4 SwiGLU layer (K and I
 *        multiples of 64, 256..3072) runs the block-scaled kernels: x and the f16 h enter
 *        the MMA as eight E2M1 digit planes (base-4 digits under one E8M0 scale per 32
 *        elements and plane), which sum to each value exactly for elements no more than
 *        2^8 (x) or 2^5 (h) below their block's largest, and within 2^-16 of that largest
 *        for the rest
 *   o_tj = w[t,j] * (h . W2[e]^T + b2[e])                    (fp32)
 *   y_t  = sum_{j=0..k-1} o_tj, in order of j, rounded to bf16 RNE.
 * x: [T_rows, K] bf16 (BF16 and MXFP4_W4A16 modes).  topk_w [T_rows, k]; the alignment
 * arrays come from moe_align over T_rows rows with the same block_m and cap_tokens.
 * y: [T_real, K] bf16.  K and I must be multiples of 32 (and of 16 output rows).
 * MXFP8 (SwiGLU only): x is E4M3 codes [T_rows, K] with x_scale [T_rows, K/32] E8M0, the
 * weights E4M3 with E8M0 scales; h is computed in fp32 and quantised to MXFP8 by the rule of
 * moe_mx_quantize before GEMM2, whose operands are then MXFP8 on both sides.  Below the
 * tensor-memory threshold (or for shapes the block-scaled kernel does not take: I or K not
 * a multiple of 128) this mode needs I <= K.  No pair-count-dependent split of K is
 * made and every output row depends only on its own input row, so padded and unpadded
 * calls give bit-identical real rows. */
moe_status moe_forward(const moe_weights* W, const void* x, const uint8_t* x_scale,
                       int64_t T_rows, int64_t T_real, int32_t k,
                       const float* topk_w, const int32_t* sorted_token_ids,
                       const int32_t* expert_ids, const int32_t* num_tokens_post_padded,
                       const int32_t* expert_offsets, int32_t block_m, int64_t cap_tokens,
                       void* y, const moe_ctx* ctx);

/* Size of the fixed device scratch array used by moe_forward_no_alloc (16 MiB). */
#define MOE_NO_ALLOC_SCRATCH_BYTES ((size_t)16 << 20)

/* moe_forward without a caller workspace; the pages have no counterpart to this call.
 *
 * For callers that cannot call cudaMalloc: code embedded in a host program that owns
 * every device allocation (it hands the plug-in its input and output buffers only), or
 * threads that must not enter the CUDA allocator, which can synchronise the device and
 * fail under memory pressure.  Arguments and results are exactly those of moe_forward;
 * ctx->workspace and ctx->workspace_bytes are ignored.  The scratch (h, o and the f16
 * copy of x) lives in a file-scope device array of MOE_NO_ALLOC_SCRATCH_BYTES inside
 * the library; every GPU that loads the library holds it until the process exits.
 *  - A call whose moe_forward_workspace_size exceeds the array returns MOE_ERR_CAPACITY
 *    (e.g. the 64-token, 2880/2880, top-4 layer needs about 4.8 MB and fits).
 *  - Every call looks up the array's device address on the current device
 *    (cudaGetSymbolAddress).  The first call on a device also loads the library's device
 *    code there; make that first call before any stream capture.
 *  - An empty batch (T_rows == 0) returns MOE_OK, as moe_forward does; invalid arguments
 *    are reported by moe_forward's own checks.
 *  - Every call shares the one array, which keeps the last call's contents.  Nothing in
 *    it has to start at zero: each call writes every scratch element it reads.  Calls
 *    that can overlap on the GPU (other streams, other host threads) race on the array:
 *    serialise them.
 *  - The call itself allocates no memory (no cudaMalloc, cudaFree or allocating library
 *    routine). */
moe_status moe_forward_no_alloc(const moe_weights* W, const void* x, const uint8_t* x_scale,
                                int64_t T_rows, int64_t T_real, int32_t k,
                                const float* topk_w, const int32_t* sorted_token_ids,
                                const int32_t* expert_ids,
                                const int32_t* num_tokens_post_padded,
                                const int32_t* expert_offsets, int32_t block_m,
                                int64_t cap_tokens, void* y, const moe_ctx* ctx);

/* ------------------------------------------------------------------------------------ *
 * One grouped GEMM over all experts in a single launch ([AITER] Summary: moe_gemm_mxfp8) *
 * ------------------------------------------------------------------------------------ */

/* Workspace bytes that let moe_grouped_gemm run W4A16 (MOE_Q_MXFP4_W4A16) weights on the
 * tensor cores: above 256 token rows the tcgen05 kernel reads A as float16, and the call
 * converts A into the workspace first (rows x Kin x 2 bytes, rows = T*k if a_per_pair else
 * T), followed by one bit per output tile that marks tiles whose weight scales need the
 * exact second pass (see moe_forward).  0 for the other modes, for T <= 256, or for invalid
 * sizes. */
size_t moe_grouped_gemm_workspace_size(moe_quant quant, int64_t T, int32_t k, int32_t N, int32_t Kin,
                                       int32_t a_per_pair);

/* out[p, :] = A[src(p), :] . W[e_p]^T + bias[e_p]   for every pair p < T*k, in bf16 RNE.
 * A: [T, Kin] (a_per_pair == 0, src = p / k) or [T*k, Kin] (a_per_pair != 0, src = p);
 *    bf16 for MOE_Q_BF16 / MOE_Q_MXFP4_W4A16, E4M3 bytes + a_scale [rows, Kin/32] E8M0
 *    for MOE_Q_MXFP8.
 * W: [E, N, Kin] (MXFP4: [E, N, Kin/2] bytes) + w_scale [E, N, Kin/32]; bias [E, N] bf16
 *    or NULL.  out: [T*k, N] bf16, indexed by pair.
 * N must be a multiple of 16 and Kin of 32.
 * Kernels: MXFP8 above 256 token rows runs the block-scaled tensor-core kernel (K and N
 * multiples of 128); bf16 above 256 rows the same tcgen05 kernel with bf16 operands (block_m
 * 128, K a multiple of 64, N of 128); W4A16 above 256 rows runs the tcgen05 kernel with
 * decoded weights in tensor memory when ctx->workspace holds
 * moe_grouped_gemm_workspace_size() bytes (block_m 128, Kin a multiple of 64; |A| <= 65504,
 * else MOE_ERR_RANGE in dev_status); every other call runs the weight-streaming kernel,
 * which needs no workspace.  The kernel
 * choice depends on T only through the bucket value 256, and each kernel reduces K in one
 * fixed order. */
moe_status moe_grouped_gemm(moe_quant quant, int32_t E, int32_t N, int32_t Kin,
                            const void* a, const uint8_t* a_scale, int32_t a_per_pair,
                            const void* w, const uint8_t* w_scale, const void* bias,
                            int64_t T, int32_t k,
                            const int32_t* sorted_token_ids, const int32_t* expert_ids,
                            const int32_t* num_tokens_post_padded, int32_t block_m,
                            int64_t cap_tokens, void* out, const moe_ctx* ctx);

/* ------------------------------------------------------------------------------------ *
 * MXFP8 quantisation (the step between the GEMMs of an MXFP8 layer)                      *
 * ------------------------------------------------------------------------------------ */

/* x [rows, cols] fp32 (cols a multiple of 32) -> codes [rows, cols] E4M3 and scales
 * [rows, cols / 32] E8M0, per 32 consecutive values of a row, by the OCP microscaling rule
 * for E4M3 elements: e = floor(log2(max |v|)) - 8 clamped to [-127, 127] (-127 for an
 * all-zero block), scale byte e + 127, code = E4M3(v / 2^e) rounded to nearest even and
 * saturated at 448, signs (zero included) kept.  A block holding a NaN gets scale 0xFF and
 * codes 0x7F.  [AITER] Summary gives the GEMM operands this format (moe_gemm_mxfp8); the
 * rule itself is the reading this library takes where the pages stop.  moe_forward applies
 * it to h in MXFP8 mode. */
moe_status moe_mx_quantize(const float* x, int64_t rows, int32_t cols, uint8_t* codes, uint8_t* scales,
                           const moe_ctx* ctx);

/* ------------------------------------------------------------------------------------ *
 * Per-token FP8 grouped GEMM over group sizes ([AITER] Summary: moe_gemm_per_token)      *
 * ------------------------------------------------------------------------------------ */

/* The rows of a are grouped by expert in expert order: expert e owns rows
 * O_e .. O_e + group_sizes[e] - 1, O_e = group_sizes[0] + ... + group_sizes[e-1]. For each
 * such row m:
 *   out[m, n] = bf16 RNE( (sum_k a[m, k] * w[e, n, k]) * a_scale[m] * w_scale[e] + bias[e, n] )
 * with the dot product of the E4M3 codes accumulated in fp32 before either scale.
 * a: [M, K] E4M3 codes; a_scale: [M] fp32; w: [E, N, K] E4M3; w_scale: [E] fp32;
 * bias: [E, N] bf16 or NULL; group_sizes: [E] int32 in device memory; out: [M, N] bf16.
 * Rows past the sum of the group sizes are not written.  Negative sizes, or sizes adding up
 * to more than M, set MOE_ERR_CAPACITY in ctx->dev_status (the sizes are read as clamped to
 * the M rows).  Limits: 1 <= E <= 1024, N and K multiples of 128, M < 2^31,
 * E * N < 2^31.  Needs no workspace. */
moe_status moe_gemm_per_token(int32_t E, int32_t N, int32_t K, const uint8_t* a, const float* a_scale,
                              const uint8_t* w, const float* w_scale, const void* bias,
                              const int32_t* group_sizes, int64_t M, void* out, const moe_ctx* ctx);

/* ------------------------------------------------------------------------------------ *
 * Weight gradient ([AITER] Summary: moe_wgrad; Tests & Benchmarks)                      *
 * ------------------------------------------------------------------------------------ */

/* Workspace bytes for moe_wgrad's slot-ordered copies (cap_tokens x N and cap_tokens x Kin
 * bf16) and the experts' block ranges (E x 2 int32), each 256-byte aligned: mode 0 with N a
 * multiple of 128, Kin of 64, block_m of 64 and E <= 1024; 0 otherwise (moe_wgrad then
 * needs none). */
size_t moe_wgrad_workspace_size(int32_t E, int32_t N, int32_t Kin, int32_t block_m, int64_t cap_tokens,
                                int32_t mode);

/* dW[e] = sum over pairs p routed to e of grad[p, :]^T (outer) input[src(p), :], fp32
 * accumulation, read straight from the alignment outputs (sentinel slots add nothing).
 * grad: [T*k, N] bf16 indexed by pair; input: [T, Kin] bf16 (input_per_pair == 0,
 * src = p / k) or [T*k, Kin] (input_per_pair != 0, src = p).  dW: [E, N, Kin] fp32.
 * mode 0: deterministic -- every dW[e] is written, zeros for experts with no pair, and
 *         repeated calls give identical bits.
 * mode 1: accumulate -- the library zeroes dW, then adds token-chunk partial sums with
 *         atomics (summation order varies between runs).
 * N and Kin must be multiples of 64.  Needs no workspace; with ctx->workspace holding
 * moe_wgrad_workspace_size() bytes, mode 0 first copies grad and input rows into slot order
 * there and the tensor-core kernel loads whole stages of them by TMA -- the same sums in the
 * same order, so the same bits as without a workspace. */
moe_status moe_wgrad(const void* grad, const void* input, int32_t input_per_pair,
                     int64_t T, int32_t k, int32_t E, int32_t N, int32_t Kin,
                     const int32_t* sorted_token_ids, const int32_t* expert_ids,
                     const int32_t* num_tokens_post_padded, int32_t block_m,
                     int64_t cap_tokens, float* dW, int32_t mode, const moe_ctx* ctx);

/* ------------------------------------------------------------------------------------ *
 * Router losses (training)                                                               *
 * ------------------------------------------------------------------------------------ */

/* Workspace bytes of moe_router_loss (0 for E outside [1, 1024]). */
size_t moe_router_loss_workspace_size(int32_t E);

/* Balance loss and z loss of a top-k softmax router, per-expert counts and the gradient of
 * the logits.  With n the tokens whose token_mask byte is not 0 (all T where it is NULL), c_e
 * the number of their choices topk_ids that name expert e, p_t = softmax(logits_t) over the E
 * experts and lse_t = log sum_e exp(logits_te):
 *   balance = sum_e f_e P_e,  f_e = E c_e / (n k),  P_e = (1/n) sum_t p_te
 *   z       = (1/n) sum_t lse_t^2
 *   loss[0] = balance_coef * balance + z_coef * z (a part of coefficient 0 is left out);
 *   loss[1] = balance;  loss[2] = z
 *   d_logits_te = (balance_coef/n) p_te (f_e - sum_e' f_e' p_te') + (2 z_coef/n) lse_t p_te
 *               + sum_{j: id_tj = e} w_tj (dw_tj - sum_i w_ti dw_ti)
 * (the counts are constants of the gradient).  The last line, the gradient through the routing
 * weights of moe_align, is there when d_topk_w is not NULL: w_tj = topk_w[t, j], dw_tj =
 * d_topk_w[t, j].
 * logits [T, E] fp32 (-inf: an expert the token may not use); topk_ids [T, k] int32, topk_w and
 * d_topk_w [T, k] fp32 (topk_w is read only with d_topk_w); token_mask [T] bytes or NULL.  counts [E] int32,
 * prob_mean [E] fp32 (P) and d_logits [T, E] fp32 may each be NULL; loss [3] fp32.  d_logits
 * may be logits itself.
 *  - A token with mask 0 counts for nothing and its row of d_logits is zeros, whatever its
 *    logits, ids and weights hold.  With no token at all every output is 0.
 *  - A row whose logits are all -inf adds its choices to the counts and nothing else; its row
 *    of d_logits is zeros.
 *  - A choice outside [0, E) of a token that counts sets MOE_ERR_INVALID_EXPERT in
 *    ctx->dev_status and is left out (of c, and of the gradient through the weights).
 * Sums and gradients in fp32, in a fixed order: repeated calls give identical bits.
 * Limits: 1 <= k <= 32, k <= E <= 1024, T*k < 2^31. */
moe_status moe_router_loss(const float* logits, const int32_t* topk_ids, const float* topk_w,
                           const float* d_topk_w, const uint8_t* token_mask, int64_t T, int32_t k, int32_t E,
                           float balance_coef, float z_coef, int32_t* counts, float* prob_mean, float* loss,
                           float* d_logits, const moe_ctx* ctx);

/* ------------------------------------------------------------------------------------ *
 * Expert activation with an 8-bit checkpoint (training)                                  *
 * ------------------------------------------------------------------------------------ */

/* Forward: gu [rows, N1] bf16 pre-activations (MOE_ACT_SWIGLU: N1 = 2I, columns 0..I-1 gate,
 * I..2I-1 up; MOE_ACT_RELU2: N1 = I) -> h [rows, I] bf16 = row_w * silu(gate) * up (or row_w *
 * max(gu, 0)^2), computed in fp32 from gu and rounded once; and the checkpoint that the backward
 * pass reads in place of gu: codes [rows, N1] E4M3 and scales [rows, N1/32] E8M0, the MXFP8
 * values of gu by the rule of moe_mx_quantize.  row_w [rows] fp32 (a pair's routing weight; NULL:
 * 1).  h may be NULL (checkpoint only).  A row of weight exactly 0 is left out: gu is not read,
 * its h and its checkpoint are zeros.  I must be a multiple of 32. */
moe_status moe_act_checkpoint(const void* gu, const float* row_w, int64_t rows, int32_t I, int32_t activation,
                              void* h, uint8_t* codes, uint8_t* scales, const moe_ctx* ctx);

/* Backward, from the checkpoint's values g, u (or z) and dh [rows, I] bf16, the gradient of h:
 *   SwiGLU: d_gu = (row_w dh u s (1 + g (1 - s)) | row_w dh g s), s = sigmoid(g);
 *   relu^2: d_gu = 2 row_w dh max(z, 0)                            [rows, N1] bf16
 *   h = row_w a, a = silu(g) u or max(z, 0)^2                       [rows, I] bf16, or NULL: the
 *       activations again, the operand of the next layer's weight gradient (moe_wgrad)
 *   d_row_w = sum_i dh_i a_i                                        [rows] fp32, or NULL: the
 *       gradient of the routing weight (moe_router_loss takes it as d_topk_w)
 * in fp32, each rounded once; the sum runs in a fixed order.  A row of weight exactly 0 is left
 * out: its outputs are zeros, whatever dh and the checkpoint hold -- d_row_w too, which loses
 * nothing where the weights are a softmax (its gradient takes d_row_w times the weight), but keeps
 * a weight that is trained by itself at 0 once it is there. */
moe_status moe_act_backward(const uint8_t* codes, const uint8_t* scales, const void* dh, const float* row_w,
                            int64_t rows, int32_t I, int32_t activation, void* d_gu, void* h, float* d_row_w,
                            const moe_ctx* ctx);

/* ------------------------------------------------------------------------------------ *
 * Dense matrix product with bias, activation and residual                                *
 * ------------------------------------------------------------------------------------ */

#define MOE_W_NK 0 /* w [N1, K]: a layer's forward weight                                  */
#define MOE_W_KN 1 /* w [K, N1]: contracted over its rows, e.g. dx = dz . W with the forward
                      weight of a layer of K outputs and N inputs                          */

/* out = act(x . W^T + bias) + residual_scale * residual
 * x [M, K] bf16; w bf16 in layout w_layout; bias [N1] bf16 or NULL; residual [M, N] in out's
 * type or NULL; out [M, N] bf16 (out_f32 == 0) or fp32.  activation: MOE_ACT_NONE or
 * MOE_ACT_RELU2 (N1 = N), or MOE_ACT_SWIGLU (N1 = 2N: gate features 0..N-1, up N..2N-1;
 * silu(gate) * up).  Everything after the products is in fp32 and rounded once.  residual may be
 * out itself (accumulation in place); out must not overlap x or w.
 * Limits: K a multiple of 8; w_layout MOE_W_KN: N a multiple of 8; M, N1, K < 2^30.  Any M
 * (0: nothing is done) and, for MOE_W_NK, any N.  An output depends on its own row of x only
 * and is summed in one fixed order for given M, N, K (which choose the kernel): repeated calls
 * give identical bits.  Needs no workspace.
 * Backward: dx = moe_dense_gemm(dz, w, the other layout), with the residual path's gradient as
 * residual; dW = moe_wgrad with E = 1 and k = 1; the bias's gradient: moe_dense_bias_grad. */
moe_status moe_dense_gemm(const void* x, const void* w, int32_t w_layout, const void* bias, const void* residual,
                          float residual_scale, int64_t M, int32_t N, int32_t K, int32_t activation, void* out,
                          int32_t out_f32, const moe_ctx* ctx);

/* d_bias[n] = sum_m dz[m, n]: dz [M, N] bf16, d_bias [N] fp32, summed in fp32 in a fixed order.
 * M = 0 gives zeros.  Needs no workspace. */
moe_status moe_dense_bias_grad(const void* dz, int64_t M, int32_t N, float* d_bias, const moe_ctx* ctx);

/* ------------------------------------------------------------------------------------ *
 * Sum of a token's pair rows                                                             *
 * ------------------------------------------------------------------------------------ */

/* y[t] = sum_{j<k} o[t*k + j] (+ residual[t]): o [T*k, K] bf16 pair rows as moe_grouped_gemm
 * writes them, residual [T, K] bf16 or NULL, y [T, K] bf16; summed in fp32 in the order of j, the
 * residual last, rounded once.  The training counterpart of moe_forward's combine: outputs whose
 * pairs carry their routing weight already (moe_act_checkpoint's row_w), and input gradients.
 * y may be residual.  K a multiple of 8, 1 <= k <= 1024, T*k < 2^31. */
moe_status moe_pair_sum(const void* o, const void* residual, int64_t T, int32_t k, int32_t K, void* y,
                        const moe_ctx* ctx);

/* ------------------------------------------------------------------------------------ *
 * Residual addition with dropout, and RMS norm                                           *
 * ------------------------------------------------------------------------------------ */

#define MOE_SCALES_NONE 0 /* no 8-bit output                                              */
#define MOE_SCALES_MX 1   /* E8M0 bytes [T, K/32]: x_scale of the MXFP8 calls             */
#define MOE_SCALES_ROW 2  /* fp32 [T]: a_scale of moe_gemm_per_token                      */

/* Dropout of the calls below.  It applies to x: element i (of the flat tensor) is dropped if its
 * 16-bit number is below d = round(65536 p) (at most 65535), else multiplied by 65536 / (65536 - d)
 * in fp32.  The number is half of a word of Philox 4x32-10 (Salmon, Moraes, Dror and Shaw, SC 2011):
 * key words rng[0] mod 2^32 and rng[0] / 2^32, counter words (b mod 2^32, b / 2^32, rng[1] mod 2^32,
 * rng_stream) with b = i / 8; word (i mod 8) / 2, its low half for even i.  rng (a seed and a step)
 * lies in device memory, so that a captured call draws other numbers once the program has changed it
 * there; forward and backward are given the same numbers in it.  rng_stream tells the dropouts of a
 * model apart. */
typedef struct {
  float p;              /* probability, 0 <= p < 1; 0: no dropout, rng is not read        */
  const int64_t* rng;   /* device [2]: seed, step                                         */
  uint32_t rng_stream;
} moe_dropout;

/* Rows that count (token_mask[t] != 0, or all where it is NULL):
 *   s = residual + dropout(x)                              -> stream [T, K], rounded once
 *   n = s * (mean_k s^2 + eps)^(-1/2) * weight             (fp32, from s before its rounding)
 *   out = n in bf16;  codes, scales = n in E4M3: MOE_SCALES_MX by the rule of moe_mx_quantize,
 *   MOE_SCALES_ROW with scale = max(max_k |n| / 448, 2^-120) and codes of n / scale
 * x [T, K] bf16 or NULL (nothing is added); residual [T, K] in the stream's type or NULL (zeros), one
 * of the two at least; token_mask [T] bytes or NULL; weight [K] bf16; stream [T, K] bf16
 * (stream_f32 == 0) or fp32, or NULL; out [T, K] bf16 or NULL; codes [T, K] and scales as the scale
 * mode says (MOE_SCALES_NONE: both NULL).  dropout may be NULL (none).
 *  - Rows that do not count may hold anything (they may be fetched, nothing of them is used); their rows
 *    of stream, out and codes are zeros and their scales those of a row of zeros (bytes 0, or 2^-120).
 *  - A NaN or an infinity in s leaves NaN in its row: row scales NaN with codes 0x7F, MX NaN in the
 *    blocks that hold a NaN n.  Sums of squares above fp32's range (|s| near 10^18) give n = 0.
 *  - stream may be residual, and out may be x; other overlaps are not allowed.
 * Limits: K a multiple of 8 (MOE_SCALES_MX: of 32), K <= 16384, T < 2^31, eps > 0 and finite.  T = 0:
 * nothing is done.  Needs no workspace. */
moe_status moe_residual_norm(const void* x, const void* residual, const uint8_t* token_mask, const void* weight,
                             int64_t T, int32_t K, float eps, const moe_dropout* dropout, int32_t stream_f32, void* stream,
                             void* out, uint8_t* codes, void* scales, int32_t scale_mode, const moe_ctx* ctx);

/* Workspace bytes of moe_residual_norm_backward with d_weight (0 for K outside its limits). */
size_t moe_residual_norm_workspace_size(int32_t K);

/* From the stream s as moe_residual_norm stored it, r = (mean_k s^2 + eps)^(-1/2), g = d_out * weight:
 *   ds = r (g - s r^2 mean_k(g s)) + d_stream
 *   d_residual = ds;  d_x = ds where x was kept, times its factor, and 0 where it was dropped
 *   d_weight = sum_t d_out s r
 * d_out [T, K] bf16: the gradient of out (and of the values that codes stand for); d_stream [T, K] in
 * the stream's type: what reaches the stream from behind, or NULL; d_residual [T, K] in the stream's
 * type, d_x [T, K] bf16 and d_weight [K] fp32 may each be NULL.  In fp32, rounded once; d_weight is
 * summed in a fixed order: repeated calls on a device give identical bits.  Rows whose sum of squares is
 * above fp32's range have ds = d_stream and add nothing to d_weight.  Rows that do not count may
 * hold anything, add nothing to d_weight, and their rows of d_residual and d_x are zeros.  d_residual may
 * be d_stream, and d_x may be d_out; other overlaps are not allowed.  Limits as above; d_weight needs
 * moe_residual_norm_workspace_size(K) bytes of workspace (T = 0 gives zeros). */
moe_status moe_residual_norm_backward(const void* d_out, const void* d_stream, const void* stream,
                                      const uint8_t* token_mask, const void* weight, int64_t T, int32_t K, float eps,
                                      const moe_dropout* dropout, int32_t stream_f32, void* d_residual, void* d_x,
                                      float* d_weight, const moe_ctx* ctx);

/* ------------------------------------------------------------------------------------ *
 * Low-rank adapters of many requests beside a dense product                              *
 * ------------------------------------------------------------------------------------ */

/* Workspace bytes of moe_adapter_gemm for M rows of R requests and rank r (0 for sizes it refuses). */
size_t moe_adapter_gemm_workspace_size(int64_t M, int32_t R, int32_t r);

/* For the rows m of request i (row_offsets[i] <= m < row_offsets[i+1]) and its adapter l = adapter[i]:
 *   out[m] = base[m] + scale[l] * (x[m] . a[l]^T) . b[l]^T      (l >= 0)
 *   out[m] = base[m]                                            (l = -1: no adapter)
 * x [M, K] bf16; a [L, r, K] bf16; b [L, N, r] bf16 (an adapter of a lower rank has zeros in the rest);
 * scale [L] fp32 or NULL (1); row_offsets [R+1] and adapter [R] int32 in device memory; base [M, N] in
 * out's type or NULL (zeros), it may be out itself: the output of moe_dense_gemm with the shared weight,
 * say; out [M, N] bf16 (out_f32 == 0) or fp32.  Rows of no request (before row_offsets[0], or from
 * row_offsets[R] on) are not written, and may hold anything, as x may in requests without an adapter.
 * Products and sums in fp32 -- x . a^T enters the second product as a sum of bf16 numbers, within 2^-17
 * of itself (2^-25 for fp32 outputs) -- rounded once; out must not overlap x, a or b.  A row depends on
 * its own request's adapter alone, also where another's is not finite.  Sums run in one fixed order for
 * given sizes, offsets and adapters: repeated calls give identical bits.
 * Data errors in ctx->dev_status: offsets that decrease or leave [0, M] (MOE_ERR_CAPACITY; such a request
 * has no rows, and the rows of requests that overlap, or that start below an offset before theirs, are
 * undefined), adapters outside [-1, L) (MOE_ERR_INVALID_EXPERT; read as -1).
 * More than 1024 requests, and adapters of 2^31 rows and more, run on the kernels for few rows a request,
 * however long they are (moe_adapter_gemm_plan): 131072 rows of 1025 requests of rank 16, 4096 -> 4096, take
 * 1.12 ms, of 1024 requests 0.69 ms, so a batch of many long requests is better given in several calls.
 * Limits: K and N multiples of 8, r a multiple of 8 up to 128, M, N, K, R < 2^30, L >= 1.  M = 0 or R = 0:
 * nothing is done.  Needs moe_adapter_gemm_workspace_size() bytes of workspace. */
moe_status moe_adapter_gemm(const void* x, const void* a, const void* b, const float* scale, const int32_t* row_offsets,
                            const int32_t* adapter, const void* base, int64_t M, int32_t N, int32_t K, int32_t r,
                            int32_t L, int32_t R, void* out, int32_t out_f32, const moe_ctx* ctx);

/* ------------------------------------------------------------------------------------ *
 * Diagnostics: failure detection of the bounded waits                                    *
 * ------------------------------------------------------------------------------------ */

/* Self-test switch of the tensor-memory kernels' failure detection (their waits on
 * mbarriers are bounded and report MOE_ERR_TIMEOUT instead of hanging).  With stall_ns > 0,
 * every later launch of the W4A16 and MXFP8 tensor-memory grouped GEMMs in this process
 * (moe_forward above 256 rows, moe_grouped_gemm in MXFP8), of moe_dense_gemm and of moe_adapter_gemm's
 * kernels for long requests runs with its copy and MMA roles
 * switched off: the other roles wait on barriers that nothing arrives on, give up after
 * stall_ns nanoseconds, write MOE_ERR_TIMEOUT to ctx->dev_status, free their tensor memory
 * and return; no copy or MMA is in flight when they give up, and the context stays usable.
 * Outputs of calls made meanwhile are undefined.  stall_ns <= 0 restores normal operation
 * (2 s limits).  Process-wide; not for use while other threads run the library.  The pages
 * have no counterpart to this call. */
void moe_debug_stall_tensor_kernels(int64_t stall_ns);

/* How moe_dense_gemm runs a product of this size on the current device, in plan[8]:
 *   plan[0] = 0: the kernel of CTA pairs (tiles of 256 x 256); the rest is 0
 *   plan[0] = 1: the kernel for few tiles; plan[1] rows of x in a tile, plan[2] weight tiles of
 *     128 features in it, plan[3] CTAs that share K, plan[4] accumulators a share is split
 *     over, plan[5] blocks of 64 of K in a stage, plan[6] rows that leave at a time, plan[7]
 *     stages
 * The same limits as moe_dense_gemm's, and M >= 1; both weight layouts run alike.  Nothing is
 * launched.  Tests and measurements use it to say which kernel they ran. */
moe_status moe_dense_gemm_plan(int64_t M, int32_t N, int32_t K, int32_t activation, int32_t out_f32, int32_t* plan);

/* Which kernels moe_adapter_gemm runs a call of this size on, in *plan: 0 those for few rows a request, 1
 * those for long requests.  The same limits as moe_adapter_gemm's, and M, R >= 1.  Nothing is launched. */
moe_status moe_adapter_gemm_plan(int64_t M, int32_t N, int32_t K, int32_t r, int32_t L, int32_t R, int32_t* plan);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */
