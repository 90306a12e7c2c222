/*
 * swiglu_mlp.h -- C ABI of the fused SwiGLU MLP library for MI355X (gfx950).
 *
 * The operation (page "[RFC] Full-pipeline SwiGLU MLP with forward/backward
 * co-optimization", Liger-Kernel issue #1347, section "Summary"):
 *
 *   forward   G = X Wg, U = X Wu, A = SiLU(G) * U, Y = A Wd
 *   backward  dA = dY Wd^T (never stored), dU = dA * SiLU(G),
 *             dG = dA * U * SiLU'(G), dWd = A^T dY,
 *             [dWg | dWu] = X^T [dG | dU]   (one GEMM),
 *             dI = [dG | dU] [Wg | Wu]^T    (one accumulator over 2H)
 *   no-grad   the forward without keeping G and U.
 *
 * Shapes and layouts. All matrices are dense and row-major (last index
 * contiguous): X, Y, dY, dX are [T, D]; Wg, Wu, dWg, dWu are [D, H];
 * Wd, dWd are [H, D]. All tensors of one call share one dtype. T >= 0 is any
 * value below 2^31; D and H must be positive multiples of 8, at most 4194296
 * for bf16/fp16 and 2097144 for fp32 (the kernels address a 256-row tile of
 * any operand with 32-bit byte offsets), and every launch's tile count must
 * fit in 32 bits. Every pointer must be 16-byte aligned; pointers to buffers
 * of zero bytes (T = 0) may be NULL.
 *
 * Numerics. bf16/fp16 storage with fp32 accumulation; every stored value is
 * rounded once (round to nearest even) from fp32. The SwiGLU epilogue is the
 * one-round program of "Scope one-round FP32 SwiGLU to the exact Qwen3.5
 * contract" (xorl PR #51, review thread): A = rnd(SiLU(g) * u), evaluated in
 * fp32 from the stored (rounded) g and u (the _ex entry points can select
 * the historical two-round program instead). SWIGLU_FP32 is true IEEE fp32:
 * fp32 operands enter the matrix cores unrounded (the TF32 issue described
 * in "[RFC] Testing Methodology for FP32 Convergence Tests on Fused
 * SwiGLU/dSwiGLU Kernels", Liger-Kernel issue #1383, section "Root Cause").
 *
 * Saved buffer. One allocation of swiglu_mlp_saved_bytes() bytes holding three
 * [T, H] planes in the order A, G, U ("store A, G, and U in one contiguous
 * buffer", issue #1347, section "Summary"). swiglu_mlp_bwd overwrites the G
 * and U planes with dG and dU ("overwrite expired G/U storage with dG/dU",
 * same section), so a saved buffer supports exactly one backward (same page,
 * section "Known limitations and validation gaps"). The A plane is left
 * unchanged.
 *
 * Ownership and streams. The caller owns every buffer; the library keeps no
 * per-call state and allocates no device memory in these calls. Work is
 * enqueued on `stream` (a hipStream_t; NULL = the default stream) and the
 * calls return before it finishes. Arguments are validated on the host
 * before anything is launched: a nonzero status means nothing was enqueued,
 * except SWIGLU_ERR_LAUNCH (a launch failed after validation). NaN and Inf
 * propagate through the arithmetic; there are no device-side traps.
 * Gradients are written (beta = 0), not accumulated.
 */
#ifndef SWIGLU_MLP_H
#define SWIGLU_MLP_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SWIGLU_BF16 = 0, /* bfloat16 storage, fp32 accumulation */
  SWIGLU_FP16 = 1, /* float16 storage, fp32 accumulation (issue #1347, "Validation environment") */
  SWIGLU_FP32 = 2  /* IEEE fp32 storage and products */
} swiglu_dtype_t;

typedef enum {
  SWIGLU_OK = 0,
  SWIGLU_ERR_NULL = 1,      /* a required pointer is NULL */
  SWIGLU_ERR_SHAPE = 2,     /* T < 0, D or H <= 0, not a multiple of 8 or above the limit, or a size overflows */
  SWIGLU_ERR_DTYPE = 3,     /* unknown dtype */
  SWIGLU_ERR_ALIGN = 4,     /* a pointer is not 16-byte aligned */
  SWIGLU_ERR_ALIAS = 5,     /* an output overlaps an input or another output */
  SWIGLU_ERR_WORKSPACE = 6, /* workspace NULL or smaller than required */
  SWIGLU_ERR_DEVICE = 7,    /* current device is not gfx950, or a HIP query failed */
  SWIGLU_ERR_LAUNCH = 8,    /* a kernel launch failed (work may be partially enqueued) */
  SWIGLU_ERR_FLAGS = 9,     /* unknown bits in the flags of an _ex entry point */
  SWIGLU_ERR_SCRATCH = 10,  /* swiglu_mlp_infer_noalloc: the call needs more than its fixed scratch */
  SWIGLU_ERR_ARG = 11       /* norms, linear layer: unknown activation or form, eps negative or not a number,
                               a bias where there is none */
} swiglu_status_t;

/* Flags of the _ex entry points (swiglu_mlp_fwd_ex, swiglu_mlp_bwd_ex,
 * swiglu_mlp_infer_ex, swiglu_mlp_infer_noalloc).
 *
 * SWIGLU_FLAG_TWO_ROUND selects the historical two-round SwiGLU program of
 * "Scope one-round FP32 SwiGLU to the exact Qwen3.5 contract" (xorl PR #51,
 * review thread): A = rnd(rnd(SiLU(g)) * u), SiLU(g) rounded to the storage
 * dtype before the product. This gives byte compatibility with unfused
 * pipelines that store SiLU(g) first. The page reports that about 27% of
 * bf16 outputs differ from the one-round program. Only A changes: G, U and
 * the backward are as without the flag, and the backward's dWd uses the A it
 * finds in the saved buffer (the backward ignores the flag). In SWIGLU_FP32
 * the two programs coincide.
 *
 * SWIGLU_FLAG_LINEAR_WEIGHTS: the weights (and the weight gradients the
 * backward writes) are in the layout of the nn.Linear layers of the
 * transformers MLP modules ("an interchangeable layer which has identical
 * __init__ and forward signatures as hf/transformers xxxMLP", maintainers'
 * thread on the mirror of issue #1347, "Three levels of APIs"):
 * Wg = gate_proj.weight and Wu = up_proj.weight are [H, D], Wd =
 * down_proj.weight is [D, H], all row-major; dWg, dWu are then [H, D] and
 * dWd is [D, H]. The kernels read this layout directly (no transposed
 * copy). The forward, backward and no-grad call of one computation must
 * all pass the same layout flag. */
#define SWIGLU_FLAG_TWO_ROUND 1u
#define SWIGLU_FLAG_LINEAR_WEIGHTS 2u
#define SWIGLU_FLAGS_ALL 3u

/* Bytes of the saved A|G|U buffer: 3 * T * H * sizeof(dtype). 0 on bad args. */
size_t swiglu_mlp_saved_bytes(int64_t T, int64_t H, int dtype);

/* Bytes of the no-grad workspace: the A plane, T * H * sizeof(dtype) ("a
 * dedicated no-grad path that does not save G/U", issue #1347, "Summary";
 * the page's table "Inference, BF16, B=1" equals A + Y at S = 256). For
 * bf16/fp16 with 1 <= T <= 128 (weight streaming) it also holds, after A and
 * 256-byte aligned, one arrival counter per 64 columns of the down
 * projection and the fp32 partial sums of its K splits, capped so that
 * workspace + Y stays within 3 (A + Y) (D = 4096, H = 11008, T = 128:
 * 10.2 MB against A + Y = 3.9 MB). The size covers both weight layouts
 * (with SWIGLU_FLAG_LINEAR_WEIGHTS only the A plane is used). 0 on bad
 * args. */
size_t swiglu_mlp_infer_workspace_bytes(int64_t T, int64_t D, int64_t H, int dtype);

/* Bytes of the backward workspace: fp32 partial tiles (256 x 256, 256 KiB
 * each) of the weight-gradient GEMMs (K = T; bf16/fp16, T > 512). Their
 * 256 x 256 output tiles run whole in rounds of one per CU of the current
 * device; the tiles of a partly filled last round are split over K when
 * that is modelled to be faster (for example D = 4096, H = 11008: 176 tiles
 * of dWd in 4 pieces, 176 MiB). 0 when no tile is split (whole
 * rounds, as at D = 4096, H = 8192) and for fp32. 0 on bad args. */
size_t swiglu_mlp_bwd_workspace_bytes(int64_t T, int64_t D, int64_t H, int dtype);

/* Forward for training. Reads X, Wg, Wu, Wd; writes Y [T, D] and the saved
 * A|G|U buffer (swiglu_mlp_saved_bytes bytes). Y and saved must not overlap
 * each other or any input. Kernels: gate/up GEMM with the fused SwiGLU
 * epilogue, then the down projection. */
int swiglu_mlp_fwd(const void* X, const void* Wg, const void* Wu, const void* Wd,
                   void* Y, void* saved, int64_t T, int64_t D, int64_t H,
                   int dtype, hipStream_t stream);

/* swiglu_mlp_fwd with epilogue flags (SWIGLU_FLAG_*); flags = 0 is
 * swiglu_mlp_fwd. Unknown bits: SWIGLU_ERR_FLAGS, nothing launched. */
int swiglu_mlp_fwd_ex(const void* X, const void* Wg, const void* Wu, const void* Wd,
                      void* Y, void* saved, int64_t T, int64_t D, int64_t H,
                      int dtype, unsigned flags, hipStream_t stream);

/* Full backward. Reads dY, X, Wg, Wu, Wd and the saved buffer written by
 * swiglu_mlp_fwd with the same inputs; writes dX [T, D] (the page's dI),
 * dWg, dWu [D, H], dWd [H, D]. Consumes the saved buffer: its G and U planes
 * hold dG and dU afterwards, and a second call on it computes garbage.
 * workspace (>= swiglu_mlp_bwd_workspace_bytes() bytes, contents on entry
 * irrelevant) may be NULL when that size is 0. Outputs and workspace must
 * not overlap each other, the inputs, or the saved buffer. */
int swiglu_mlp_bwd(const void* dY, const void* X, const void* Wg, const void* Wu,
                   const void* Wd, void* saved, void* dX, void* dWg, void* dWu,
                   void* dWd, void* workspace, size_t workspace_bytes,
                   int64_t T, int64_t D, int64_t H, int dtype, hipStream_t stream);

/* swiglu_mlp_bwd with flags (SWIGLU_FLAG_*); flags = 0 is swiglu_mlp_bwd.
 * With SWIGLU_FLAG_LINEAR_WEIGHTS the weights are read, and dWg, dWu, dWd
 * written, in the nn.Linear layout. Unknown bits: SWIGLU_ERR_FLAGS, nothing
 * launched. */
int swiglu_mlp_bwd_ex(const void* dY, const void* X, const void* Wg, const void* Wu,
                      const void* Wd, void* saved, void* dX, void* dWg, void* dWu,
                      void* dWd, void* workspace, size_t workspace_bytes,
                      int64_t T, int64_t D, int64_t H, int dtype, unsigned flags,
                      hipStream_t stream);

/* No-grad forward: Y [T, D] from X and the weights; G and U are never
 * stored. workspace (>= swiglu_mlp_infer_workspace_bytes bytes) holds A and,
 * for T <= 128, counters and partial sums; its contents on entry do not
 * matter (the call clears what it counts on). Two launches. Calls that use
 * one workspace must not overlap (stream order them). Y must not overlap
 * the inputs or the workspace. */
int swiglu_mlp_infer(const void* X, const void* Wg, const void* Wu, const void* Wd,
                     void* Y, void* workspace, size_t workspace_bytes,
                     int64_t T, int64_t D, int64_t H, int dtype, hipStream_t stream);

/* swiglu_mlp_infer with epilogue flags (SWIGLU_FLAG_*); flags = 0 is
 * swiglu_mlp_infer. Unknown bits: SWIGLU_ERR_FLAGS, nothing launched. */
int swiglu_mlp_infer_ex(const void* X, const void* Wg, const void* Wu, const void* Wd,
                        void* Y, void* workspace, size_t workspace_bytes,
                        int64_t T, int64_t D, int64_t H, int dtype, unsigned flags,
                        hipStream_t stream);

/* Allocation-free no-grad forward, for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc). Same computation, kernels and results as
 * swiglu_mlp_infer_ex with the same flags, but the workspace is a fixed
 * array of SWIGLU_NOALLOC_SCRATCH_BYTES inside the library: one copy per
 * device, held from the library's first call on that device until the
 * process ends. Calls allocate nothing (no hipMalloc, hipFree or allocating
 * library routine). A call whose swiglu_mlp_infer_workspace_bytes exceeds
 * the scratch returns SWIGLU_ERR_SCRATCH with nothing launched (bf16 at
 * D = 4096, H = 11008: every T <= 128, and T <= 1524 above that). The
 * caller passes the inputs and Y as for swiglu_mlp_infer. Every call on one
 * device shares that device's scratch, which keeps the last call's
 * contents (the call clears what it counts on): calls that overlap on one
 * device race and must be ordered (one stream, or events). */
#define SWIGLU_NOALLOC_SCRATCH_BYTES (32u << 20)
int swiglu_mlp_infer_noalloc(const void* X, const void* Wg, const void* Wu, const void* Wd,
                             void* Y, int64_t T, int64_t D, int64_t H, int dtype,
                             unsigned flags, hipStream_t stream);

/* ---- Serving with few tokens ----------------------------------------------
 * A mixture of SwiGLU experts and products with 4-bit weights, for the calls
 * whose time is that of reading the weights (a decoding step: one token per
 * sequence). No backward. All weights are in the nn.Linear layout; sums are
 * fp32, A is rounded once to the storage type between the two launches, Y
 * once at the end. For few tokens (T <= 8, or up to 2 choices per expert on
 * average; 4-bit weights 4 and 1) a 16-bit A also keeps what its rounding left,
 * so that its values may reach twice the type's largest; else those past the
 * range are infinities. Any T up to SWIGLU_FEW_MAX_T is computed, in chunks of
 * 64 tokens that each read the weights they need again; the kernels are meant
 * for T up to about 64. T = 0 passes the checks and does nothing. Infinities
 * and NaN stay with their token and have the values of the formulas.
 *
 * Router (swiglu_mlp_moe_route): logits l = X Wr^T over E experts, the k
 * largest of each token in descending order (equal logits: the lower index
 * first; NaN before everything), weights softmax(l) over all E, divided by
 * the chosen ones' sum when `renorm` is nonzero. X [T, D], Wr [E, D] in one
 * dtype; weights fp32 (from the fp32 logits: about 3e-7 relative) and ids int32
 * [T, k], 4-byte aligned. The order is that of the exact logits: those closer to
 * a neighbour than the fp32 sums can tell apart are summed again in fp64 (among
 * the 64 leading ones of a token).
 *
 * Experts (swiglu_mlp_moe_experts): Y[t] = sum_j weights[t][j] *
 * ((SiLU(X[t] Wg_e^T) * (X[t] Wu_e^T)) Wd_e^T), e = ids[t][j]; Wg, Wu
 * [E, H, D], Wd [E, D, H]. An id outside [0, E) chooses nothing (a dropped or
 * padded token, an expert of another device); a token without a choice gets
 * zeros. A token may choose one expert more than once. swiglu_mlp_moe_infer
 * is the router and the experts in one call (the choices stay in the
 * workspace). 1 <= k <= min(E, 32), E <= 1024, D and H multiples of 8 up to
 * SWIGLU_FEW_MAX_D.
 *
 * 4-bit weights (bf16 and fp16 storage): W[n][k] = scale[n][k / group] *
 * (code[n][k] - zero[n][k / group]), codes 0..15, group 32, 64 or 128
 * dividing K, N a multiple of 8; zero = 8 where there are no zero points.
 * The kernels read a packed layout that swiglu_mlp_w4_pack writes once from
 * codes [X][N][K/2] (two to a byte, the even k in the low half), scales
 * [X][N][K/group] in the storage type and zeros [X][N][K/group] bytes (or
 * NULL). swiglu_mlp_w4_quantize makes codes, scales and, where zeros is not
 * NULL, zero points from a 16-bit W [X][N][K] (a NaN makes its group's scale
 * NaN); swiglu_mlp_w4_dequantize writes the packed weight back as rows (for a
 * long prompt, whose products are bound by arithmetic). Products are exact per
 * code and scaled in fp32: no weight is rounded. */
#define SWIGLU_FEW_MAX_T 65536
#define SWIGLU_FEW_MAX_D 131072

typedef struct {
  const void* data; /* swiglu_mlp_w4_bytes() bytes written by swiglu_mlp_w4_pack */
  int64_t experts;  /* matrices: 1 for a dense weight */
  int64_t N, K;     /* out_features, in_features */
  int32_t group;
  int32_t has_zeros;
} swiglu_w4_t;

/* workspace: the logits' partial sums. Contents on entry do not matter. 0 bytes
 * on bad args. */
size_t swiglu_mlp_moe_route_workspace_bytes(int64_t T, int64_t D, int64_t E, int dtype);
int swiglu_mlp_moe_route(const void* X, const void* Wr, float* weights, int32_t* ids, void* workspace,
                         size_t workspace_bytes, int64_t T, int64_t D, int64_t E, int64_t k, int renorm,
                         int dtype, hipStream_t stream);

/* Bytes of a mixture's workspace: the A plane [T k, H], the arrival counters
 * and fp32 partial sums of the down projection where its K is split over
 * workgroups (before them, in the same place, the router's workspace), and
 * the router's weights and ids, each 256-byte aligned.
 * Contents on entry do not matter; calls that share one must be
 * stream-ordered. 0 on bad args. */
size_t swiglu_mlp_moe_workspace_bytes(int64_t T, int64_t D, int64_t H, int64_t E, int64_t k, int dtype);

int swiglu_mlp_moe_experts(const void* X, const float* weights, const int32_t* ids, const void* Wg,
                           const void* Wu, const void* Wd, void* Y, void* workspace,
                           size_t workspace_bytes, int64_t T, int64_t D, int64_t H, int64_t E,
                           int64_t k, int dtype, hipStream_t stream);
int swiglu_mlp_moe_infer(const void* X, const void* Wr, const void* Wg, const void* Wu, const void* Wd,
                         void* Y, void* workspace, size_t workspace_bytes, int64_t T, int64_t D,
                         int64_t H, int64_t E, int64_t k, int renorm, int dtype, hipStream_t stream);
int swiglu_mlp_moe_experts_w4(const void* X, const float* weights, const int32_t* ids,
                              const swiglu_w4_t* Wg, const swiglu_w4_t* Wu, const swiglu_w4_t* Wd,
                              void* Y, void* workspace, size_t workspace_bytes, int64_t T, int64_t k,
                              int dtype, hipStream_t stream);
int swiglu_mlp_moe_infer_w4(const void* X, const void* Wr, const swiglu_w4_t* Wg,
                            const swiglu_w4_t* Wu, const swiglu_w4_t* Wd, void* Y, void* workspace,
                            size_t workspace_bytes, int64_t T, int64_t k, int renorm, int dtype,
                            hipStream_t stream);

/* Bytes of a packed weight (0 on bad args). */
size_t swiglu_mlp_w4_bytes(int64_t experts, int64_t N, int64_t K, int group, int has_zeros);
int swiglu_mlp_w4_quantize(const void* W, void* codes, void* scales, void* zeros, int64_t experts,
                           int64_t N, int64_t K, int group, int dtype, hipStream_t stream);
int swiglu_mlp_w4_pack(const void* codes, const void* scales, const void* zeros, void* data,
                       int64_t experts, int64_t N, int64_t K, int group, hipStream_t stream);
int swiglu_mlp_w4_dequantize(const swiglu_w4_t* w, void* W, int dtype, hipStream_t stream);

/* Y [T, N] = X [T, K] W^T. One launch; with more than 16 tokens and few output
 * columns two, and a workspace of partial sums between them (0 bytes
 * otherwise; may be NULL then). */
size_t swiglu_mlp_w4_linear_workspace_bytes(int64_t T, int64_t N, int64_t K, int dtype);
int swiglu_mlp_w4_linear(const void* X, const swiglu_w4_t* w, void* Y, void* workspace,
                         size_t workspace_bytes, int64_t T, int dtype, hipStream_t stream);

/* The dense block with 4-bit weights, two launches; workspace: A [T, H], then
 * counters and partial sums as a mixture's. The three weights share group
 * size and have zero points all or none. */
size_t swiglu_mlp_w4_infer_workspace_bytes(int64_t T, int64_t D, int64_t H, int dtype);
int swiglu_mlp_w4_infer(const void* X, const swiglu_w4_t* Wg, const swiglu_w4_t* Wu,
                        const swiglu_w4_t* Wd, void* Y, void* workspace, size_t workspace_bytes,
                        int64_t T, int dtype, hipStream_t stream);

/* ---- Norms and the linear layer -------------------------------------------
 * What stands before and beside the block in the same models, for training
 * and for inference.
 *
 * Norms over the last axis of X [T, D] (rms = 0: layer norm, 1: RMS norm):
 *   n = (x - mean) rstd, y = n weight + bias, rstd = 1 / sqrt(mean((x - mean)^2) + eps)
 * and for RMS norm the same with mean = 0 and no bias. Sums are fp32, the
 * variance that of the differences from the mean, the mean corrected by theirs
 * (a row of one number has it as its mean); squares past fp32's range
 * are infinities. Any D from 1 to SWIGLU_NORM_MAX_D; pointers need the alignment
 * of an element only (workspace: 16 bytes). stats, [2][T] (mean, rstd; RMS
 * norm [T], rstd) in fp32, is what the backward needs; NULL without one.
 * The backward writes dX (plus dres where that is not NULL: the gradient
 * that reaches x past the norm, as in x + f(norm(x))), dweight and dbias (NULL:
 * not wanted). The sums over tokens have a fixed order. T = 0 writes zero
 * weight gradients. workspace: fp32 parts of those sums; contents on entry do
 * not matter. */
#define SWIGLU_NORM_MAX_D 1048576
size_t swiglu_mlp_norm_stats_bytes(int64_t T, int rms);
size_t swiglu_mlp_norm_bwd_workspace_bytes(int64_t T, int64_t D, int rms, int dtype);
int swiglu_mlp_norm_fwd(const void* X, const void* weight, const void* bias, void* Y, float* stats,
                        int64_t T, int64_t D, float eps, int rms, int dtype, hipStream_t stream);
int swiglu_mlp_norm_bwd(const void* dY, const void* X, const void* weight, const float* stats,
                        const void* dres, void* dX, void* dweight, void* dbias, void* workspace,
                        size_t workspace_bytes, int64_t T, int64_t D, int rms, int dtype,
                        hipStream_t stream);

/* Linear layer with its epilogue: Z = X W^T + bias, Y = act(Z) + residual. X
 * [T, K], W [N, K] (nn.Linear layout), bias [N], residual, Y, Z [T, N]; bias,
 * residual and Z may be NULL. T, N and K as T, D and H above. Z is the fp32 sum
 * rounded to the storage type, kept for the backward; Y comes from the fp32
 * sum itself and is rounded once. At most 64 tokens stream the weight.
 * The backward reads dY, X, W and, where there is an activation, Z, and
 * writes dX = dZ W, dW = dZ^T X and dbias = sum over tokens of dZ, where dZ =
 * dY act'(Z) (rounded to the storage type for the two products, not for the
 * sum); NULL: not wanted, and X may be NULL where dW is, W where dX is. The
 * residual's gradient is dY. T = 0 writes zero
 * weight gradients. gelu is z Phi(z), gelu_tanh its form with tanh; relu's
 * derivative at 0 and at NaN is 0, every derivative at an infinity its limit (a
 * Z past the storage type's range). In bf16 and fp16 silu and gelu_tanh of values
 * below about -87 (2u for gelu_tanh) may be a zero. workspace contents on entry do
 * not matter; calls that share one must be stream-ordered. */
typedef enum {
  SWIGLU_ACT_NONE = 0,
  SWIGLU_ACT_RELU = 1,
  SWIGLU_ACT_GELU = 2,
  SWIGLU_ACT_GELU_TANH = 3,
  SWIGLU_ACT_SILU = 4
} swiglu_act_t;
#define SWIGLU_NUM_ACTS 5
size_t swiglu_mlp_linear_workspace_bytes(int64_t T, int64_t N, int64_t K, int dtype);
int swiglu_mlp_linear_fwd(const void* X, const void* W, const void* bias, const void* residual, void* Y,
                          void* Z, void* workspace, size_t workspace_bytes, int64_t T, int64_t N,
                          int64_t K, int act, int dtype, hipStream_t stream);
size_t swiglu_mlp_linear_bwd_workspace_bytes(int64_t T, int64_t N, int64_t K, int act, int dtype);
int swiglu_mlp_linear_bwd(const void* dY, const void* X, const void* W, const void* Z, void* dX, void* dW,
                          void* dbias, void* workspace, size_t workspace_bytes, int64_t T, int64_t N,
                          int64_t K, int act, int dtype, hipStream_t stream);

/* How a linear layer of these sizes runs on the current device (launches nothing;
 * for profiles and tests). engine: 0 stream of the weight, 1 tiles of 64 x 64, 2 of
 * 64 x 128, 3 of 128 x 128, 4 ring of 256 x 256 tiles; parts: of the summed axis.
 * dw, dx: whether the backward is asked for them; neither: the forward. The
 * entries of what is not asked for are 0; `together`: both gradients in one launch. */
typedef struct {
  int32_t fwd_engine, fwd_parts, dw_engine, dw_parts, dx_engine, dx_parts, together;
} swiglu_linear_plan_t;
int swiglu_mlp_linear_plan(int64_t T, int64_t N, int64_t K, int dtype, int dw, int dx,
                           swiglu_linear_plan_t* plan);

/* Static description of a status code (never NULL). */
const char* swiglu_mlp_status_string(int status);

/* ---- Profiling aid (not part of the computation) -------------------------
 * Stage ids, one per kernel of the path:
 *   0 gate/up GEMM + SwiGLU (fwd)      1 down projection (fwd)
 *   2 dA GEMM + in-place dSwiGLU       3 dWd = A^T dY
 *   4 [dWg | dWu] = X^T [dG | dU]      5 dI single accumulator
 *   6 no-grad gate/up (A only)         7 no-grad down projection
 *   8 stages 3 + 2 in one launch       9 stages 4 + 5 in one launch
 *  10 router                          11 few-token gate/up (experts, 4-bit)
 *  12 few-token down projection or 4-bit product
 *  13 norm                            14 norm's backward
 *  15 linear layer                    16 its dZ and dbias
 *  17 its dX                          18 its dW
 * (bf16/fp16 run every stage as its own launch; in fp32 with T > 512 the
 * backward runs as launches 8 and 9, where the long-K weight-gradient tiles
 * are dispatched first and the short tiles of the other stage fill in
 * behind them.)
 * swiglu_mlp_timer_start(capacity) makes every later launch of a stage record
 * a HIP event pair around it on the launch stream, up to `capacity` launches
 * per stage (events are created here; returns a status). swiglu_mlp_timer_stop
 * waits for the recorded events and writes, for each of the first `n` stages,
 * the summed milliseconds to ms[s] and the launch count to count[s], then
 * disables recording. Not thread-safe; meant for a benchmark's timed loop. */
#define SWIGLU_NUM_STAGES 19
int swiglu_mlp_timer_start(int capacity);
int swiglu_mlp_timer_stop(double* ms, int* count, int n);

#ifdef __cplusplus
}
#endif
#endif /* SWIGLU_MLP_H */
