/*
 * ls_reduce.h -- C ABI of libls_reduce.so: fused softmax and LayerNorm reduce
 * kernels of a Transformer layer (forward and backward) for NVIDIA GB300
 * (sm_103a).
 *
 * The operations are the LightSeq-style reduce kernels described on the pages
 *   "CMU 11-868 L10: Accelerating Transformers on GPUs, and Where LightSeq
 *    Finds the Time", section "Technique 2: rewrite the formula, drop a
 *    synchronization" (slides 21-26), and
 *   "CMU 11-868 HW4：把 Softmax 與 LayerNorm 寫成 CUDA 融合 kernel",
 *    section 題目結構與配分 (Problems 1.1, 1.2, 2.1, 2.2).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Pointers named as device buffers must be CUDA device (or managed) memory
 *    owned by the caller.  The library never allocates, frees or
 *    synchronises; it only enqueues kernels on `stream`.
 *  - `stream` is a cudaStream_t passed as void* (NULL = the legacy default
 *    stream).  All work is asynchronous with respect to the host.
 *  - Tensors are dense, row-major, with the last dimension contiguous.
 *  - Storage dtype `dt` applies to every `void*` tensor of a call (scores,
 *    mask, gamma, beta, activations and their gradients).  Arithmetic is FP32
 *    for every storage dtype; 16-bit outputs are rounded to nearest-even.
 *    LayerNorm statistics (mean, rstd) and the gamma/beta gradients are
 *    always FP32.
 *  - Pointers must be aligned to their element size.  Buffers that are also
 *    16-byte aligned, with a row length in bytes that is a multiple of 16,
 *    take the 128-bit vector path; all others take a scalar path of the same
 *    kernel family (same results, lower bandwidth).  There is no CPU path.
 *  - A zero-sized problem (no rows, or an empty row for softmax) is a valid
 *    no-op, except where stated.  Negative sizes, NULL required pointers,
 *    unsupported dtypes and inconsistent shapes are rejected on the host
 *    before anything is launched; nothing is written in that case.
 *  - Return value: LS_OK once the kernels are enqueued.  A launch failure
 *    reported by the CUDA runtime is LS_ERR_CUDA.  Faults that happen while
 *    the kernels run surface at the caller's next synchronisation, as for any
 *    CUDA work.
 */
#ifndef LS_REDUCE_H
#define LS_REDUCE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum ls_dtype {
    LS_F32 = 0,  /* IEEE binary32 */
    LS_F16 = 1,  /* IEEE binary16 */
    LS_BF16 = 2  /* bfloat16 */
} ls_dtype;

typedef enum ls_status {
    LS_OK = 0,
    LS_ERR_INVALID_ARG = 1,  /* NULL pointer, negative size, inconsistent shape,
                                overlapping outputs */
    LS_ERR_UNSUPPORTED = 2,  /* unknown dtype, or a size beyond the limits below */
    LS_ERR_MISALIGNED = 3,   /* pointer not aligned to its element size */
    LS_ERR_WORKSPACE = 4,    /* workspace missing or smaller than required */
    LS_ERR_CUDA = 5          /* the CUDA runtime rejected a launch */
} ls_status;

/* Largest row length (Tk for softmax, hidden for LayerNorm) accepted. */
#define LS_MAX_ROW_LENGTH ((int64_t)1 << 30)

/*
 * Attention softmax forward ("Problem 1.1" of the HW4 page; slides 23-26 of
 * the L10 page).  For every row (b, h, i) of the score tensor:
 *     z_j = -inf                       if causal and j > i + (Tk - Tq)  (future key)
 *     z_j = inp[b,h,i,j] + mask[b,j]   otherwise
 *     out[b,h,i,j] = exp(z_j - max_k z_k) / sum_k exp(z_k - max_k z_k)
 * A row whose every key is -inf is written as zeros.
 *
 *   out   [B,H,Tq,Tk] dt, device, written.  May equal `inp` (in place).
 *   inp   [B,H,Tq,Tk] dt, device, read.  Scores are expected to be finite.
 *   mask  [B,Tk] dt additive mask (0 = keep, -inf = padded key; any finite
 *         bias is added, and a row that sees only keys hidden by one, -1e10
 *         or the type's lowest value, is the softmax of its z), device,
 *         read; NULL means no mask.  Shared by all heads and queries of a
 *         batch entry.  Keys whose mask is -inf are not read from `inp` where
 *         a batch entry's visible keys are contiguous, and never matter.
 *   causal  nonzero: mask future keys.  Requires Tq <= Tk; the Tq queries are
 *           the last Tq positions of the key sequence (bottom-right
 *           alignment), so query i sees keys j <= i + (Tk - Tq); with
 *           Tq == Tk that is j <= i.
 * Errors: LS_ERR_INVALID_ARG for NULL out/inp with a non-empty problem,
 * negative sizes, or causal with Tq > Tk; LS_ERR_UNSUPPORTED for Tk beyond
 * LS_MAX_ROW_LENGTH or an unknown dtype.
 */
ls_status ls_softmax_fw(void *out, const void *inp, const void *mask,
                        int64_t B, int64_t H, int64_t Tq, int64_t Tk,
                        int causal, ls_dtype dt, void *stream);

/*
 * Attention softmax backward ("Problem 1.2" of the HW4 page).  For every
 * row:  dinp_j = out_j * (dout_j - sum_k out_k * dout_k),
 * the vector-Jacobian product of the forward softmax at its output `out_fw`.
 * Masked and future keys need no mask argument: their forward output is 0.
 *
 *   dinp    [B,H,Tq,Tk] dt, device, written.  May equal `dout`.
 *   dout    [B,H,Tq,Tk] dt, device, read (gradient of the softmax output).
 *   out_fw  [B,H,Tq,Tk] dt, device, read (the forward output).
 * Errors as for ls_softmax_fw (no causal/mask arguments here).
 */
ls_status ls_softmax_bw(void *dinp, const void *dout, const void *out_fw,
                        int64_t B, int64_t H, int64_t Tq, int64_t Tk,
                        ls_dtype dt, void *stream);

/*
 * Attention softmax backward that skips invisible keys: the same result as
 * ls_softmax_bw when `out_fw` is the forward output (0 on masked and future
 * keys), but keys that are masked (mask == -inf) or in the causal future are
 * neither read from `dout` / `out_fw` nor summed; their gradient is written
 * as 0.  Per row:
 *     s      = sum over visible k of out_k * dout_k
 *     dinp_j = out_j * (dout_j - s)   on visible keys, 0 elsewhere
 * It is the backward counterpart of ls_softmax_fw's read skipping (the L10
 * page's slide 30 names the score gradient as the O(T^2) tensor of the
 * attention backward).
 *
 *   dinp    [B,H,Tq,Tk] dt, device, written.  May equal `dout`.
 *   dout, out_fw  [B,H,Tq,Tk] dt, device, read on visible keys only.
 *   mask    [B,Tk] dt additive mask or NULL, as for ls_softmax_fw.
 *   causal  as for ls_softmax_fw (Tq <= Tk, bottom-right alignment).
 * Errors as for ls_softmax_fw.
 */
ls_status ls_softmax_bw_masked(void *dinp, const void *dout, const void *out_fw,
                               const void *mask, int64_t B, int64_t H, int64_t Tq,
                               int64_t Tk, int causal, ls_dtype dt, void *stream);

/*
 * Scaled softmax, forward: the fused "scale + mask + softmax" of an attention
 * layer (the L10 page, section "Technique 1", fuses the operations between
 * the GEMMs into custom kernels; the score scale is one of them).  As
 * ls_softmax_fw, with the scores multiplied by `scale` (e.g. 1/sqrt(head
 * dimension)) before the additive mask:
 *     z_j = scale * x_j + mask[b, j]   (-inf for causal future keys)
 *     y   = softmax(z)
 * The scale is folded into the exponent (no extra pass, no extra arithmetic
 * on unmasked chunks).  scale must be finite and > 0, else
 * LS_ERR_INVALID_ARG.  Other arguments and errors as for ls_softmax_fw;
 * ls_softmax_fw is this function with scale = 1 (bitwise).
 */
ls_status ls_softmax_fw_scaled(void *out, const void *inp, const void *mask, int64_t B,
                               int64_t H, int64_t Tq, int64_t Tk, int causal, float scale,
                               ls_dtype dt, void *stream);

/*
 * Scaled softmax, backward over the visible keys: the gradient of the scores
 * of ls_softmax_fw_scaled,
 *     dinp_j = scale * y_j * (dout_j - sum over visible k of y_k dout_k)
 * on visible keys and 0 on the others (as ls_softmax_bw_masked, which is this
 * function with scale = 1, bitwise).  scale must be finite and > 0.
 */
ls_status ls_softmax_bw_masked_scaled(void *dinp, const void *dout, const void *out_fw,
                                      const void *mask, int64_t B, int64_t H, int64_t Tq,
                                      int64_t Tk, int causal, float scale, ls_dtype dt,
                                      void *stream);

/*
 * LayerNorm forward ("Problem 2.1" of the HW4 page; slide 21 of the L10
 * page).  For every row of x [rows, hidden], the mean and variance come from
 * ONE fused reduction of the two sums sum(x') and sum(x'^2), x' = x - x_0
 * (x_0 the row's first element; the variance is shift-invariant and the
 * shift keeps the one-pass form exact for constant rows):
 *     mu   = x_0 + mean(x'),   var = max(mean(x'^2) - mean(x')^2, 0)
 *     rstd = 1 / sqrt(var + eps)
 *     y_j  = (x_j - mu) * rstd * gamma_j + beta_j
 *
 *   y      [rows, hidden] dt, device, written.
 *   mean   [rows] float32, device, written (the saved mu).
 *   rstd   [rows] float32, device, written (the saved 1/sqrt(var + eps)).
 *   x      [rows, hidden] dt, device, read.
 *   gamma, beta  [hidden] dt, device, read.
 *   eps    added to the variance inside the square root (the pages use 1e-8).
 * Errors: LS_ERR_INVALID_ARG for NULL pointers with rows > 0, negative rows,
 * hidden < 1, or eps < 0 / not finite; LS_ERR_UNSUPPORTED for hidden beyond
 * LS_MAX_ROW_LENGTH or an unknown dtype.
 */
ls_status ls_layernorm_fw(void *y, float *mean, float *rstd, const void *x,
                          const void *gamma, const void *beta, int64_t rows,
                          int64_t hidden, float eps, ls_dtype dt, void *stream);

/*
 * LayerNorm backward, input gradient ("Problem 2.2" of the HW4 page; slide
 * 22 of the L10 page: two sums computed in parallel, then elementwise work).
 * With xhat = (x - mean) * rstd and g = gamma * dy, per row:
 *     S1 = sum_j g_j,   S2 = sum_j g_j * xhat_j      (one fused reduction)
 *     dx_j = rstd * (g_j - S1 / hidden - xhat_j * S2 / hidden)
 *
 *   dx     [rows, hidden] dt, device, written.  May equal `dy`.
 *   dy     [rows, hidden] dt, device, read (gradient of y).
 *   x      [rows, hidden] dt, device, read (the forward input).
 *   gamma  [hidden] dt, device, read.
 *   mean, rstd  [rows] float32, device, read (as saved by ls_layernorm_fw).
 * Errors as for ls_layernorm_fw.
 */
ls_status ls_layernorm_bw_dinp(void *dx, const void *dy, const void *x,
                               const void *gamma, const float *mean,
                               const float *rstd, int64_t rows, int64_t hidden,
                               ls_dtype dt, void *stream);

/*
 * Bytes of device workspace ls_layernorm_bw_dgamma_dbeta needs for a
 * [rows, hidden] problem (the same for every dtype).  Returns 0 for
 * rows <= 0 or hidden <= 0.  Host-only; launches nothing.
 */
size_t ls_layernorm_bw_dgamma_dbeta_workspace_size(int64_t rows, int64_t hidden);

/*
 * LayerNorm backward, gamma and beta gradients ("Problem 2.2" of the HW4
 * page: the cross-row kernel).  Column sums over all rows:
 *     dgamma_j = sum_r dy_rj * (x_rj - mean_r) * rstd_r
 *     dbeta_j  = sum_r dy_rj
 * computed in a fixed order that depends only on (rows, hidden): the result
 * is bitwise reproducible from run to run and GPU to GPU.  With rows == 0 the
 * outputs are set to zero.
 *
 *   dgamma, dbeta  [hidden] float32, device, written (overwritten, not
 *                  accumulated into).
 *   dy, x          [rows, hidden] dt, device, read.
 *   mean, rstd     [rows] float32, device, read.
 *   workspace      device scratch of at least
 *                  ls_layernorm_bw_dgamma_dbeta_workspace_size(rows, hidden)
 *                  bytes, 16-byte aligned; its contents on entry do not
 *                  matter and are left undefined.  May be NULL when that size
 *                  is 0.  Calls that overlap on the GPU must not share it.
 * Errors as for ls_layernorm_fw, plus LS_ERR_WORKSPACE when the workspace is
 * NULL, too small or not 16-byte aligned.
 */
ls_status ls_layernorm_bw_dgamma_dbeta(float *dgamma, float *dbeta,
                                       const void *dy, const void *x,
                                       const float *mean, const float *rstd,
                                       int64_t rows, int64_t hidden,
                                       void *workspace, size_t workspace_bytes,
                                       ls_dtype dt, void *stream);

/*
 * Bytes of device workspace ls_layernorm_bw needs for a [rows, hidden]
 * problem (the same for every dtype): 8 * hidden bytes for each of at most
 * 456 partial sums, or what ls_layernorm_bw_dgamma_dbeta needs when that is
 * more (the scalar path below).  Returns 0 for rows <= 0 or hidden <= 0.
 * Host-only; launches nothing.
 */
size_t ls_layernorm_bw_workspace_size(int64_t rows, int64_t hidden);

/*
 * Fused LayerNorm backward: the input gradient of ls_layernorm_bw_dinp and the
 * gamma / beta gradients of ls_layernorm_bw_dgamma_dbeta from one read of dy
 * and x ("Problem 2.2" of the HW4 page asks for both halves of the backward;
 * slide 22 of the L10 page lists the per-row sums).  The rows are cut into
 * contiguous chunks (at most 456 for rows of one 16-byte vector, 304 for up
 * to 512 vectors, 152 for wider rows) by a rule that depends only on (rows,
 * hidden, dt); one thread block per chunk writes dx for its rows and its
 * chunk's column sums of dy * xhat and dy, and a second kernel adds the
 * chunks in index order.  dgamma and dbeta are therefore bitwise
 * reproducible from run to run and GPU to GPU; their rounding, and dx's (the
 * row sums are split across threads differently), may differ from the
 * separate kernels' in the last bits.
 *
 *   dx             [rows, hidden] dt, device, written.  May equal dy (each
 *                  row's dy is staged on chip before its dx is written).
 *   dgamma, dbeta  [hidden] float32, device, written (overwritten).
 *   dy, x          [rows, hidden] dt, device, read.
 *   gamma          [hidden] dt, device, read.
 *   mean, rstd     [rows] float32, device, read (as saved by ls_layernorm_fw).
 *   workspace      device scratch of at least
 *                  ls_layernorm_bw_workspace_size(rows, hidden) bytes,
 *                  16-byte aligned, contents ignored; may be NULL when that
 *                  size is 0.  Calls that overlap on the GPU must not share it.
 * Errors as for ls_layernorm_bw_dgamma_dbeta.  Rows wider than 2048 16-byte
 * vectors (hidden > 16384 for 16-bit storage, > 8192 for fp32), or pointers
 * or widths that are not 16-byte multiples, run the two separate kernels
 * instead, with the same results as calling them.
 */
ls_status ls_layernorm_bw(void *dx, float *dgamma, float *dbeta, const void *dy,
                          const void *x, const void *gamma, const float *mean,
                          const float *rstd, int64_t rows, int64_t hidden,
                          void *workspace, size_t workspace_bytes, ls_dtype dt,
                          void *stream);

/*
 * Size of the device array that ls_layernorm_bw_dgamma_dbeta_noalloc uses as
 * scratch (4 MiB).  It covers every problem with hidden <= 524288 (2^19),
 * whatever the row count: the partial sums take at most 456 * 2048 bytes
 * for hidden below 116736 (456 tiles of 256), and 8 * hidden bytes (one
 * row chunk) above it.
 */
#define LS_DGDB_NOALLOC_SCRATCH_BYTES ((size_t)4 << 20)

/*
 * LayerNorm gamma/beta gradients without any allocation.  The pages have no
 * counterpart to this entry point; it exists for callers that cannot hand the
 * library a workspace -- code that receives only tensor pointers and a stream
 * from a host program (a plugin, or C code with no access to the host's
 * allocator), or code that may not call cudaMalloc at that moment because
 * cudaMalloc can synchronise the device or break the host's memory budget.
 *
 * Computes exactly what ls_layernorm_bw_dgamma_dbeta computes (same kernels,
 * same fixed summation order, bitwise the same result), but keeps the partial
 * sums in a fixed device array of LS_DGDB_NOALLOC_SCRATCH_BYTES compiled into
 * the library, which every GPU that loads the library holds until the process
 * exits.  It calls no cudaMalloc, cudaFree or other allocating routine.
 *
 *   Arguments as for ls_layernorm_bw_dgamma_dbeta, without the workspace.
 *   Problems whose partial sums need more than LS_DGDB_NOALLOC_SCRATCH_BYTES
 *   (ls_layernorm_bw_dgamma_dbeta_workspace_size(rows, hidden) larger than
 *   that) are refused with LS_ERR_UNSUPPORTED before anything is launched.
 *
 * Every call looks up the array's device address (cudaGetSymbolAddress) with
 * the caller's device current; once the library's module is loaded on that
 * device the lookup is a host-side query that allocates nothing, and a fresh
 * lookup stays valid after cudaDeviceReset.  The first call on a device may
 * be the one that loads the module, which places the array in device memory
 * and can synchronise: make one call during set-up, before any stream
 * capture, if that must not happen later.  All calls on a device share the one
 * array: calls that may overlap on the GPU (different streams without
 * ordering between them) race on it and must not be issued that way.  The
 * array keeps the last call's partial sums; each call overwrites every
 * partial it reads, so nothing needs to be cleared between calls.
 */
ls_status ls_layernorm_bw_dgamma_dbeta_noalloc(float *dgamma, float *dbeta,
                                               const void *dy, const void *x,
                                               const float *mean, const float *rstd,
                                               int64_t rows, int64_t hidden,
                                               ls_dtype dt, void *stream);

/*
 * RMSNorm forward: the one-reduction LayerNorm variant of the page
 * "FastTransformer: Breaking the Compiler Ceiling via Architectural
 * Co-Design", section 5.4 "Vectorized Pre-RMSNorm" (no mean centring, no
 * bias).  Per row of x [rows, hidden]:
 *     rstd = 1 / sqrt(mean(x^2) + eps),   y_j = x_j * rstd * gamma_j
 *
 *   y      [rows, hidden] dt, device, written.
 *   rstd   [rows] float32, device, written (saved for the backward).
 *   x      [rows, hidden] dt, device, read.
 *   gamma  [hidden] dt, device, read.
 *   eps    added inside the square root (the page uses 1e-6).
 * Errors as for ls_layernorm_fw.
 */
ls_status ls_rmsnorm_fw(void *y, float *rstd, const void *x, const void *gamma, int64_t rows,
                        int64_t hidden, float eps, ls_dtype dt, void *stream);

/*
 * RMSNorm backward, input gradient.  With xhat = x * rstd and g = gamma * dy,
 * per row:  S = sum_j g_j * xhat_j,  dx_j = rstd * (g_j - xhat_j * S / hidden).
 *
 *   dx     [rows, hidden] dt, device, written.  May equal `dy`.
 *   dy, x  [rows, hidden] dt, device, read.
 *   gamma  [hidden] dt, device, read.
 *   rstd   [rows] float32, device, read (as saved by ls_rmsnorm_fw).
 * Errors as for ls_layernorm_bw_dinp.
 */
ls_status ls_rmsnorm_bw_dinp(void *dx, const void *dy, const void *x, const void *gamma,
                             const float *rstd, int64_t rows, int64_t hidden, ls_dtype dt,
                             void *stream);

/*
 * RMSNorm backward, gamma gradient: dgamma_j = sum_r dy_rj * x_rj * rstd_r,
 * in the same fixed order as ls_layernorm_bw_dgamma_dbeta (bitwise
 * reproducible).  `workspace` as for that function, sized by
 * ls_layernorm_bw_dgamma_dbeta_workspace_size(rows, hidden).
 *
 *   dgamma  [hidden] float32, device, written (overwritten).
 *   dy, x   [rows, hidden] dt, device, read.
 *   rstd    [rows] float32, device, read.
 * Errors as for ls_layernorm_bw_dgamma_dbeta.
 */
ls_status ls_rmsnorm_bw_dgamma(float *dgamma, const void *dy, const void *x, const float *rstd,
                               int64_t rows, int64_t hidden, void *workspace,
                               size_t workspace_bytes, ls_dtype dt, void *stream);

/*
 * Softmax cross entropy over a vocabulary, forward.  The L10 page, section
 * "Technique 1: kernel fusion, leaving only GEMMs to cuBLAS" (slide 12),
 * makes cross entropy the third custom reduce kernel beside LayerNorm and
 * softmax; the page gives no formula, so this is the textbook one, in FP32.
 * For each row r of logits z [rows, vocab] with target class t = target[r]:
 *     lse_r  = log sum_j exp(z_rj)        (computed as max + log sum exp(z - max))
 *     loss_r = lse_r - z_rt               (= -log softmax(z_r)_t)
 * A negative target marks an ignored row (padding): loss_r = lse_r = 0 and
 * the row is not read.  A target >= vocab gives loss_r = lse_r = NaN (there
 * is no device-side trap).  No label smoothing; one loss per row (the caller
 * reduces, e.g. sums over its non-ignored rows).
 *
 *   loss, lse  [rows] float32, device, written.
 *   logits     [rows, vocab] dt, device, read; any vocab >= 1 (rows need
 *              not start on 16-byte boundaries).
 *   target     [rows] int32, device, read.
 * Errors: LS_ERR_INVALID_ARG for rows < 0, vocab < 1 or a NULL pointer when
 * rows > 0; LS_ERR_UNSUPPORTED for an unknown dtype or vocab above
 * LS_MAX_ROW_LENGTH; LS_ERR_MISALIGNED for a pointer not aligned to its
 * element; LS_ERR_CUDA for a failed launch.  rows == 0 launches nothing.
 */
ls_status ls_cross_entropy_fw(float *loss, float *lse, const void *logits,
                              const int32_t *target, int64_t rows, int64_t vocab,
                              ls_dtype dt, void *stream);

/*
 * Softmax cross entropy, backward: the gradient of loss_r * dloss_r with
 * respect to the logits, from the lse saved by the forward:
 *     dlogits_rj = dloss_r * ( exp(z_rj - lse_r) - [j == t_r] )
 * Ignored rows (t_r < 0) are written as zeros and rows with t_r >= vocab as
 * NaN; neither is read.
 *
 *   dlogits  [rows, vocab] dt, device, written.  May equal logits.
 *   logits   [rows, vocab] dt, device, read.
 *   target   [rows] int32, device, read.
 *   lse      [rows] float32, device, read (as written by ls_cross_entropy_fw).
 *   dloss    [rows] float32, device, read (upstream gradient of each row's
 *            loss; 1 / (number of non-ignored rows) for a mean loss).
 * Errors as for ls_cross_entropy_fw.  When logits and dlogits do not sit at
 * the same offset modulo 16 bytes, every element is moved singly (slower,
 * same result).
 */
ls_status ls_cross_entropy_bw(void *dlogits, const void *logits, const int32_t *target,
                              const float *lse, const float *dloss, int64_t rows,
                              int64_t vocab, ls_dtype dt, void *stream);

/* Limits of the softmax with a relative position bias. */
#define LS_MAX_RELPOS_DISTANCE ((int64_t)2048)
#define LS_MAX_RELPOS_BUCKETS ((int64_t)65536)

/*
 * Attention softmax with a learned relative position bias by buckets,
 * forward.  The scaled softmax (ls_softmax_fw_scaled) plus one learned number
 * per (bucket of the distance from query to key, head).  The Tq queries are
 * the last Tq of the Tk key positions, so with R = max_distance:
 *     r    = min(max(j - (i + Tk - Tq), -R), R)
 *     z_ij = scale * x[b,h,i,j] + table[bucket[r + R], h] + mask[b,j]
 *     out[b,h,i,:] = softmax over the visible j of z_i
 * A key is invisible when its mask element is -inf or, with causal, when it
 * lies in the query's future (j > i + Tk - Tq); invisible keys are written as
 * 0 and their scores never matter, NaN or not.  A row without a visible key,
 * or whose every z is -inf, is written as zeros.  A single decoding step is
 * Tq = 1.  z is formed in FP32 (scaled score and bias in one rounding, then
 * the mask) and the weights are e^(z - max z) at any magnitude: a row that
 * sees only keys hidden by a finite mask is the softmax of those z.
 *
 *   out    [B,H,Tq,Tk] dt, device, written.  May equal `inp` (in place).
 *   inp    [B,H,Tq,Tk] dt, device, read.
 *   mask   [B,Tk] dt additive mask, device, read; NULL means no mask.  Any
 *          value: 0, -inf, the type's lowest value, a finite bias.
 *   table  [num_buckets,H] dt, device, read: the learned bias.
 *   bucket [2R + 1] int32, device, read: the bucket of each clipped distance
 *          -R ... R.  Ids outside [0, num_buckets) add no bias.
 *   causal, scale  as for ls_softmax_fw_scaled (Tq > Tk only without causal).
 * Errors: LS_ERR_INVALID_ARG for NULL out / inp / table / bucket with a
 * non-empty problem, negative sizes, num_buckets or max_distance < 1, causal
 * with Tq > Tk, scale not finite or <= 0; LS_ERR_UNSUPPORTED for an unknown
 * dtype or sizes beyond the limits above or LS_MAX_ROW_LENGTH (Tq and Tk).
 */
ls_status ls_softmax_fw_relpos(void *out, const void *inp, const void *mask, const void *table,
                               const int32_t *bucket, int64_t B, int64_t H, int64_t Tq,
                               int64_t Tk, int64_t num_buckets, int64_t max_distance, int causal,
                               float scale, ls_dtype dt, void *stream);

/*
 * Bytes of device workspace ls_softmax_bw_relpos needs for H heads and
 * max_distance, whatever the other sizes and the dtype.  0 for sizes that it
 * refuses.  Host-only; launches nothing.
 */
size_t ls_softmax_bw_relpos_workspace_size(int64_t H, int64_t max_distance);

/*
 * Attention softmax with a relative position bias, backward: the gradients of
 * the scores and of the table.  On visible keys, with s = sum over visible k
 * of out_k * dout_k,
 *     dz_ij      = out_ij * (dout_ij - s_i)
 *     dinp_ij    = scale * dz_ij                      (0 on invisible keys)
 *     dtable[k,h] = sum over every b, i and visible j with
 *                   bucket[r + R] == k of dz[b,h,i,j]
 * dz enters the table's sum in FP32, before dinp is rounded.  Invisible keys
 * are not summed, and what dout / out_fw hold there never matters; 16-byte
 * chunks without a visible key are not read where a batch entry's visible keys
 * are contiguous.  The sums are taken in an order that depends only on the
 * sizes, the dtype and the pointers' offsets within 16 bytes: the same call is
 * bitwise reproducible.
 *
 *   dinp    [B,H,Tq,Tk] dt, device, written.  May equal `dout`.
 *   dtable  [num_buckets,H] float32, device, written (overwritten; zeros when
 *           there is no score).
 *   dout, out_fw  [B,H,Tq,Tk] dt, device, read (see above).
 *   mask, bucket, causal, scale  as given to the forward.
 *   workspace  device scratch of at least
 *           ls_softmax_bw_relpos_workspace_size(H, max_distance) bytes,
 *           16-byte aligned, contents ignored.  May be NULL when there is no
 *           score.  Calls that overlap on the GPU must not share it.
 * Errors as for ls_softmax_fw_relpos, plus LS_ERR_WORKSPACE.
 */
ls_status ls_softmax_bw_relpos(void *dinp, float *dtable, const void *dout, const void *out_fw,
                               const void *mask, const int32_t *bucket, int64_t B, int64_t H,
                               int64_t Tq, int64_t Tk, int64_t num_buckets, int64_t max_distance,
                               int causal, float scale, void *workspace, size_t workspace_bytes,
                               ls_dtype dt, void *stream);

/* Largest head size and most query or key heads of the per-head norm. */
#define LS_MAX_HEAD_DIM ((int64_t)1024)
#define LS_MAX_HEADS ((int64_t)1 << 29)

/*
 * RMSNorm of every query head and every key head, and the rotation by the
 * token's position, in one pass (ls_rmsnorm_fw over rows of D features, with
 * one gamma for all query heads and one for all key heads).  Per row x of
 * token t:
 *     rstd = 1 / sqrt(mean(x^2) + eps),   n_j = x_j * rstd * gamma_j
 *     (y_a, y_b) = (n_a c - n_b s, n_b c + n_a s),  c = cos[positions[t], p],
 *                                                   s = sin[positions[t], p]
 * for the pairs p < rot / 2, which are (p, p + rot / 2), or (2p, 2p + 1) when
 * interleaved; y_j = n_j for j >= rot.  rot = 0 is the norm alone.
 * The normed value is not rounded before the rotation.
 *
 *   q_out, k_out  [tokens,Hq,D], [tokens,Hk,D] dt, device, written.  May equal
 *                 q and k (in place, same strides).  Any other overlap with
 *                 each other or with q and k is refused, also both in place
 *                 where q and k share memory.
 *   q_rstd, k_rstd  [tokens,Hq], [tokens,Hk] float32, device, written (saved
 *                 for the backward); NULL: not written.
 *   q, k          [tokens,Hq,D], [tokens,Hk,D] dt, device, read.
 *   *_stride      elements from one token to the next (>= heads * D; heads
 *                 and features are dense), so q and k may be slices of one
 *                 packed projection.
 *   gamma_q, gamma_k  [D] dt, device, read.
 *   cos, sin      [max_pos, rot / 2] float32, device, read.
 *   positions     [tokens] int32, device, read.  A position outside
 *                 [0, max_pos) makes the token's rotated features NaN.
 * Hq or Hk may be 0 (its pointers are then ignored).
 * Errors: LS_ERR_INVALID_ARG for a NULL pointer that is needed, negative
 * sizes, D < 1, rot odd or outside [0, D], a stride below heads * D, eps < 0
 * or not finite, overlapping outputs; LS_ERR_UNSUPPORTED for an unknown dtype or sizes beyond the
 * limits above; LS_ERR_MISALIGNED as everywhere.
 */
ls_status ls_qk_norm_rope_fw(void *q_out, void *k_out, float *q_rstd, float *k_rstd,
                             const void *q, const void *k, const void *gamma_q,
                             const void *gamma_k, const float *cos, const float *sin,
                             const int32_t *positions, int64_t tokens, int64_t Hq, int64_t Hk,
                             int64_t D, int64_t rot, int64_t max_pos, int64_t q_out_stride,
                             int64_t k_out_stride, int64_t q_stride, int64_t k_stride,
                             int interleaved, float eps, ls_dtype dt, void *stream);

/*
 * Bytes of device workspace ls_qk_norm_rope_bw needs.  0 for no tokens and
 * for sizes that it refuses.  Host-only; launches nothing.
 */
size_t ls_qk_norm_rope_bw_workspace_size(int64_t tokens, int64_t Hq, int64_t Hk, int64_t D);

/*
 * Per-head norm with rotation, backward: the gradients of q and k and of both
 * gammas, in one pass over the inputs.  With dn the upstream gradient turned
 * back by the position's angles, xhat = x * rstd and g = gamma * dn, per row:
 *     dx_j     = rstd * (g_j - xhat_j * sum_k(g_k xhat_k) / D)
 *     dgamma_j = sum over every token and head of the side of dn_j * xhat_j
 * The gamma sums are taken in an order that depends only on the sizes, the
 * dtype, the strides and the pointers' alignment (which choose the width of the
 * accesses): the same call is bitwise reproducible.
 *
 *   dq, dk        [tokens,heads,D] dt, device, written.  May equal dq_out and
 *                 dk_out (same strides); other overlaps are refused, as in the
 *                 forward.
 *   dgamma_q, dgamma_k  [D] float32, device, written (overwritten; zeros when
 *                 tokens == 0; ignored, not written, for a side of 0 heads).
 *   dq_out, dk_out  gradients of the forward's outputs, dt, device, read.
 *   q, k, gamma_*, cos, sin, positions  as given to the forward.
 *   q_rstd, k_rstd  as saved by the forward.
 *   workspace     device scratch of at least
 *                 ls_qk_norm_rope_bw_workspace_size(tokens, Hq, Hk, D) bytes,
 *                 16-byte aligned, contents ignored; may be NULL when that is
 *                 0.  Calls that overlap on the GPU must not share it.
 * A position outside the table makes the token's gradients NaN, and the
 * gamma gradients of the rotated features.  Errors as for the forward, plus
 * LS_ERR_WORKSPACE.
 */
ls_status ls_qk_norm_rope_bw(void *dq, void *dk, float *dgamma_q, float *dgamma_k,
                             const void *dq_out, const void *dk_out, const void *q, const void *k,
                             const void *gamma_q, const void *gamma_k, const float *q_rstd,
                             const float *k_rstd, const float *cos, const float *sin,
                             const int32_t *positions, int64_t tokens, int64_t Hq, int64_t Hk,
                             int64_t D, int64_t rot, int64_t max_pos, int64_t dq_stride,
                             int64_t dk_stride, int64_t dq_out_stride, int64_t dk_out_stride,
                             int64_t q_stride, int64_t k_stride, int interleaved, void *workspace,
                             size_t workspace_bytes, ls_dtype dt, void *stream);

/* Most elements of a list of gradients. */
#define LS_MAX_GRAD_ELEMENTS ((int64_t)1 << 40)

/*
 * Bytes of device workspace ls_grad_norm and ls_grad_clip need for a list of
 * `count` tensors, whatever their sizes.  Host-only; launches nothing.
 */
size_t ls_grad_norm_workspace_size(int64_t count);

/*
 * Global norm of a list of gradient tensors:
 *     norm = sqrt(sum over all tensors of the sum of g^2)
 * Squares are summed in FP32 within 8 vectors of a thread (in FP64 where they
 * would over- or underflow) and in FP64 beyond, in an order that depends only
 * on the list's sizes and dtypes and its pointers' offsets within 16 bytes: the
 * same call is bitwise reproducible.  inf or NaN elements give inf or NaN.
 *
 *   norm    [1] float32, device, written (0 for an empty list).
 *   grads, sizes, dtypes  HOST arrays of `count` entries, read before the
 *           call returns: device pointers to dense tensors, their element
 *           counts and their ls_dtype codes (types may be mixed).  A pointer
 *           needs only its element's alignment.  Tensors of 0 elements are
 *           skipped.
 *   workspace  device scratch of at least ls_grad_norm_workspace_size(count)
 *           bytes, 16-byte aligned, contents ignored; may be NULL for an
 *           empty list.  Calls that overlap on the GPU must not share it.
 * Errors: LS_ERR_INVALID_ARG for NULL pointers, negative counts or sizes;
 * LS_ERR_UNSUPPORTED for an unknown dtype or more than LS_MAX_GRAD_ELEMENTS;
 * LS_ERR_MISALIGNED; LS_ERR_WORKSPACE; LS_ERR_CUDA.
 */
ls_status ls_grad_norm(float *norm, const void *const *grads, const int64_t *sizes,
                       const int32_t *dtypes, int64_t count, void *workspace,
                       size_t workspace_bytes, void *stream);

/*
 * Clipping by the global norm: the norm as ls_grad_norm computes it, and
 *     out = g * min(1, max_norm / (norm + eps))
 * for every tensor.  In place (out[i] == grads[i]) a list that needs no
 * clipping is left as it is, unwritten.  A NaN norm makes every output NaN;
 * an infinite one makes finite elements 0 and infinite ones NaN.
 *
 *   out     HOST array of `count` device pointers, written, each of its
 *           gradient's size and dtype; may equal grads entry by entry.  Any
 *           other overlap, of two outputs or of an output and a gradient, is
 *           refused.  (Gradients may overlap one another where they are only
 *           read.)
 *   max_norm  finite and > 0.   eps  finite and >= 0.
 * Other arguments and errors as for ls_grad_norm; LS_ERR_INVALID_ARG for a
 * bad max_norm or eps and for overlapping outputs.
 */
ls_status ls_grad_clip(float *norm, void *const *out, const void *const *grads,
                       const int64_t *sizes, const int32_t *dtypes, int64_t count, float max_norm,
                       float eps, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Difference of two attention softmax maps with a learned weight, forward (the
 * attention map of a differential attention layer).  Head h of batch entry b
 * has two maps of scores over the same keys; the Tq queries are the last Tq of
 * the Tk key positions:
 *     z_aj = scale * x_a[b,h,i,j] + mask[b,j]      (a = 1, 2)
 *     p_a  = softmax over the visible j of z_a
 *     out[b,h,i,j] = p_1j - lam_h * p_2j
 * Visible and invisible keys as for ls_softmax_fw_relpos: invisible ones are
 * written as 0 and their scores never matter, NaN or not; a map without a
 * visible key, or whose every z is -inf, is 0.  NaN or +inf among a map's
 * visible scores make the row's visible outputs NaN.
 *
 *   out    [B,H,Tq,Tk] dt, dense, device, written.  May equal x1 where that is
 *          dense (in place).
 *   stats  [B,H,Tq,4] float32, 16-byte aligned, device, written: of each map
 *          the largest z (0 if there is none) and 1 / sum_j exp(z_j - largest)
 *          (0 if nothing is visible), saved for the backward; NULL: not
 *          written.
 *   x1, x2 [B,H,Tq,Tk] dt, device, read, with dense [Tq,Tk] and strides of
 *          x*_batch and x*_head elements (>= 0) between batch entries and
 *          heads: both may be slices of one tensor [B,2H,Tq,Tk], by halves or
 *          by neighbouring heads.  A stride over a single entry is ignored.
 *   lam    [lam_count] float32, device, read: one weight per head (lam_count
 *          == H) or one for all heads (lam_count == 1).
 *   mask, causal, scale  as for ls_softmax_fw_relpos; mask may be NULL.
 * Errors: LS_ERR_INVALID_ARG for NULL out / x1 / x2 / lam with a non-empty
 * problem, negative sizes or strides, lam_count other than 1 and H, causal with
 * Tq > Tk, scale not finite or <= 0, outputs that overlap each other or an
 * input (except in place); LS_ERR_UNSUPPORTED for an unknown dtype, Tq or Tk
 * beyond LS_MAX_ROW_LENGTH, H beyond LS_MAX_HEADS, B beyond 2^30 or more than
 * 2^44 rows; LS_ERR_MISALIGNED as everywhere.
 */
ls_status ls_softmax_fw_diff(void *out, float *stats, const void *x1, const void *x2,
                             const float *lam, const void *mask, int64_t B, int64_t H, int64_t Tq,
                             int64_t Tk, int64_t x1_batch, int64_t x1_head, int64_t x2_batch,
                             int64_t x2_head, int64_t lam_count, int causal, float scale,
                             ls_dtype dt, void *stream);

/*
 * Bytes of device workspace ls_softmax_bw_diff needs: 4 per row.  0 without
 * rows and for sizes that it refuses.  Host-only; launches nothing.
 */
size_t ls_softmax_bw_diff_workspace_size(int64_t B, int64_t H, int64_t Tq);

/*
 * Difference of two attention softmax maps, backward.  The weights p_a are made
 * again from the scores and the saved statistics.  On visible keys, with
 * D_a = sum over visible k of p_ak dout_k:
 *     dx_1j  =  scale * p_1j * (dout_j - D_1)
 *     dx_2j  = -scale * lam_h * p_2j * (dout_j - D_2)       (0 on invisible keys)
 *     dlam_h = -sum over b, i of D_2     (lam_count == 1: over h too)
 * Invisible keys are not summed, and what dout and the scores hold there never
 * matters.  The sums' order depends only on the sizes, the strides, the dtype
 * and the pointers' offsets within 16 bytes: the same call is bitwise
 * reproducible.
 *
 *   dx1, dx2  as x1 and x2, written, with strides of their own; no two heads
 *           may share memory.  dx1 may equal x1 and dx2 x2 (same strides).
 *   dlam    [lam_count] float32, device, written (overwritten; zeros when there
 *           is no score).
 *   dout    [B,H,Tq,Tk] dt, dense, device, read on visible keys.
 *   x1, x2, lam, mask, causal, scale  as given to the forward.
 *   stats   as written by the forward.
 *   workspace  device scratch of at least
 *           ls_softmax_bw_diff_workspace_size(B, H, Tq) bytes, 16-byte aligned,
 *           contents ignored.  May be NULL when there is no score.  Calls that
 *           overlap on the GPU must not share it.
 * Errors as for ls_softmax_fw_diff, plus LS_ERR_WORKSPACE.
 */
ls_status ls_softmax_bw_diff(void *dx1, void *dx2, float *dlam, const void *dout, const void *x1,
                             const void *x2, const float *lam, const float *stats,
                             const void *mask, int64_t B, int64_t H, int64_t Tq, int64_t Tk,
                             int64_t dx1_batch, int64_t dx1_head, int64_t dx2_batch,
                             int64_t dx2_head, int64_t x1_batch, int64_t x1_head, int64_t x2_batch,
                             int64_t x2_head, int64_t lam_count, int causal, float scale,
                             void *workspace, size_t workspace_bytes, ls_dtype dt, void *stream);

/* Widest row of the norms around a block. */
#define LS_MAX_BLOCK_HIDDEN ((int64_t)16384)

/*
 * Norms after and before a block of a Transformer layer, with the block's gate
 * and the scaled residual stream, forward.  x is the block's output, r the
 * residual stream it is added to; N is LayerNorm (layer != 0) or RMSNorm:
 *     n = N(x; gamma_post, beta_post)          or x without gamma_post
 *     h = residual_scale * r + gate * n        (gate 1 without gate)
 *     y = N(h; gamma_pre, beta_pre)            only with gamma_pre
 *   LayerNorm: N(v)_j = (v_j - mean) * rstd * gamma_j + beta_j
 *   RMSNorm:   N(v)_j = v_j * rstd * gamma_j
 * rstd = 1 / sqrt(variance (mean square for RMSNorm) + eps).  h enters its norm
 * in FP32, before it is rounded.
 *
 *   h      [rows, hidden] dt, device, written: the new residual stream.
 *   y      [rows, hidden] dt, device, written: the next block's input; ignored
 *          without gamma_pre.  h and y may each be x or r itself.
 *   stats  [4, rows] float32, device, written: mean and rstd of x, mean and
 *          rstd of h (mean 0 for RMSNorm; 0 and 1 for a norm that is not taken).
 *   x, r   [rows, hidden] dt, device, read.
 *   gate   [gates, hidden] dt, device, read, or NULL: rows [k * rows / gates,
 *          (k + 1) * rows / gates) share gate k, so one gate is a learned vector,
 *          one per sequence a conditioned one, `rows` of them one per token.
 *   gamma_post, beta_post, gamma_pre, beta_pre  [hidden] dt, device, read, or
 *          NULL; a beta wants LayerNorm and its gamma.
 * Errors: LS_ERR_INVALID_ARG for negative rows, hidden < 1, NULL h / stats / x
 * / r or (with gamma_pre) y when rows > 0, gates < 1 or no divisor of rows, a
 * beta without LayerNorm or gamma, eps < 0 or not finite, residual_scale not
 * finite, overlapping outputs; LS_ERR_UNSUPPORTED for an unknown dtype, hidden
 * beyond LS_MAX_BLOCK_HIDDEN or more than 2^40 rows; LS_ERR_MISALIGNED as
 * everywhere.
 */
ls_status ls_block_norm_fw(void *h, void *y, float *stats, const void *x, const void *r,
                           const void *gate, const void *gamma_post, const void *beta_post,
                           const void *gamma_pre, const void *beta_pre, int64_t rows,
                           int64_t hidden, int64_t gates, float residual_scale, float eps,
                           int layer, ls_dtype dt, void *stream);

/*
 * Bytes of device workspace ls_block_norm_bw needs (gates: 0 without a gate).
 * 0 without rows and for sizes that it refuses.  Host-only; launches nothing.
 */
size_t ls_block_norm_bw_workspace_size(int64_t rows, int64_t hidden, int64_t gates, int layer,
                                       ls_dtype dt);

/*
 * Norms around a block, backward.  With up = dh + (input gradient of the second
 * norm for dy), xhat and hhat the normed rows before gamma:
 *     dr = residual_scale * up
 *     dx = input gradient of the first norm for gate * up   (gate * up without it)
 *     dgate_k     = sum over the gate's rows of up * n
 *     dgamma_post = sum of gate * up * xhat,   dbeta_post = sum of gate * up
 *     dgamma_pre  = sum of dy * hhat,          dbeta_pre  = sum of dy
 * The sums are taken in FP32 in an order that depends only on the sizes and the
 * dtype: the same call is bitwise reproducible.
 *
 *   dx, dr  [rows, hidden] dt, device, written.  dx may be dy, dh, x or h
 *          itself, dr dy, dh or h.
 *   dgate  [gates, hidden] float32, device, written; ignored without gate.
 *   dgamma_post, dgamma_pre  [hidden] float32, device, written; ignored without
 *          the gamma.  dbeta_post, dbeta_pre  [hidden] float32, device, written,
 *          or NULL; want LayerNorm and the gamma.  All sums are zeros when rows
 *          == 0.
 *   dy     [rows, hidden] dt, device, read with gamma_pre: gradient of y.
 *   dh     [rows, hidden] dt, device, read: gradient of h from its other uses;
 *          NULL (with gamma_pre): none.
 *   x      as given to the forward; read with gamma_post or gate.
 *   h, stats  as written by the forward (h read with gamma_pre).
 *   gate, gamma_post, beta_post, gamma_pre  as given to the forward.  (beta_post
 *          only enters dgate, which is that of a forward without it where it is
 *          left out: no status tells.)
 *   workspace  device scratch of at least ls_block_norm_bw_workspace_size(...)
 *          bytes, 16-byte aligned, contents ignored; may be NULL when that is 0.
 *          Calls that overlap on the GPU must not share it.
 * Errors as for the forward (dy and h missing with gamma_pre, dh missing
 * without it, x missing with gamma_post or gate, a missing gradient of a given
 * parameter), plus LS_ERR_WORKSPACE.
 */
ls_status ls_block_norm_bw(void *dx, void *dr, float *dgate, float *dgamma_post, float *dbeta_post,
                           float *dgamma_pre, float *dbeta_pre, const void *dy, const void *dh,
                           const void *x, const void *h, const float *stats, const void *gate,
                           const void *gamma_post, const void *beta_post, const void *gamma_pre,
                           int64_t rows, int64_t hidden, int64_t gates, float residual_scale,
                           int layer, void *workspace, size_t workspace_bytes, ls_dtype dt,
                           void *stream);

/* Limits of the cross entropy from hidden states. */
#define LS_MAX_LINEAR_ROWS ((int64_t)1 << 26)
#define LS_MAX_LINEAR_HIDDEN ((int64_t)1 << 16)
#define LS_MAX_LINEAR_VOCAB ((int64_t)1 << 28)

/*
 * Bytes of device workspace the cross entropy from hidden states needs, with R
 * the rows up to a multiple of 256, D hidden up to a multiple of 8, and 2 bytes an
 * element of a copy (fp32: 6, three planes):
 *   both      a copy of the rows that count, R D elements; for fp32 and where
 *             hidden is no multiple of 8 a copy of w, vocab D elements; up to
 *             16 bytes per row beside them
 *   forward   16 bytes per row of R and 256 vocabulary entries
 *   backward  the logits' gradients of a piece of the vocabulary, R times as many
 *             elements as it has entries (all of it where that takes up to
 *             512 MiB, else as much as does, 4096 entries at least); where dx is
 *             summed over pieces or cuts of them 4 R D bytes for each cut, at
 *             most 32 (cut are the sums of few rows over a large vocabulary)
 * 0 for sizes that are refused and, forward, without rows.  Host-only; launches
 * nothing.
 */
size_t ls_linear_cross_entropy_fw_workspace_size(int64_t rows, int64_t hidden, int64_t vocab,
                                                 ls_dtype dt);
size_t ls_linear_cross_entropy_bw_workspace_size(int64_t rows, int64_t hidden, int64_t vocab,
                                                 ls_dtype dt);

/*
 * Softmax cross entropy taken from hidden states and the vocabulary matrix,
 * forward: ls_cross_entropy_fw of the logits z = x w^T, which are never stored.
 * For each row r with target class t = target[r]:
 *     lse_r  = log sum_v exp(z_rv),   loss_r = lse_r - z_rt
 * The logits are FP32 sums of exact products of the stored values (fp32: of
 * products good to about 2^-23) and are not rounded to the storage type; the
 * tensor cores cut a sum off every 16 products, and parts of it are added
 * rounding to nearest (up to about 2^-17 of a sum of terms of one sign).
 * Ignored rows (negative target): loss = lse = 0; target >= vocab: NaN; neither
 * row of x is read.
 * No wait inside the kernels lasts longer than two seconds of wall-clock time:
 * what hung on one that ran out (the GPU was taken away for so long) comes out as
 * NaN, in both directions, without a status.
 *
 *   loss, lse  [rows] float32, device, written.
 *   x          [rows, hidden] dt, device, read.
 *   w          [vocab, hidden] dt, device, read.  16-byte aligned where its
 *              rows are 16-bit types of a multiple of 8 elements.
 *   target     [rows] int32, device, read.
 *   workspace  device scratch of at least
 *              ls_linear_cross_entropy_fw_workspace_size(...) bytes, 16-byte
 *              aligned, contents ignored.  Calls that overlap on the GPU must
 *              not share it.
 * Errors: LS_ERR_INVALID_ARG for rows < 0, hidden or vocab < 1, a NULL pointer
 * when rows > 0, outputs or a workspace that overlap each other or an input;
 * LS_ERR_UNSUPPORTED for an unknown dtype, sizes beyond the limits above or
 * more than 2^38 elements in x and w; LS_ERR_MISALIGNED, LS_ERR_WORKSPACE,
 * LS_ERR_CUDA as everywhere.  rows == 0 launches nothing.
 */
ls_status ls_linear_cross_entropy_fw(float *loss, float *lse, const void *x, const void *w,
                                     const int32_t *target, int64_t rows, int64_t hidden,
                                     int64_t vocab, void *workspace, size_t workspace_bytes,
                                     ls_dtype dt, void *stream);

/*
 * Softmax cross entropy from hidden states, backward: the gradients of
 * sum_r loss_r * dloss_r, from the lse saved by the forward.
 *     q_rv = dloss_r * ( exp(z_rv - lse_r) - [v == t_r] ),  0 in ignored rows
 *     dx   = q w,     dw = q^T x
 * q is made and used by pieces of the vocabulary.  For 16-bit types each q is
 * rounded once to the storage type (fp16: after a scaling by a power of two
 * that keeps small weights normal), since the tensor cores multiply operands
 * of one type; sums are FP32.  Ignored rows get dx = 0 and add nothing to dw,
 * whatever x, lse and dloss hold there.  A target >= vocab makes its row of dx
 * and all of dw NaN.  The sums' order depends only on the sizes, the dtype and
 * the targets' signs: the same call is bitwise reproducible.
 *
 *   dx         [rows, hidden] dt, device, written.
 *   dw         [vocab, hidden] dt, device, written (overwritten; zeros when no
 *              row counts); NULL: not computed.
 *   x, w, target  as given to the forward.
 *   lse, dloss [rows] float32, device, read.
 *   workspace  as for the forward, ls_linear_cross_entropy_bw_workspace_size.
 * Errors as for the forward.
 */
ls_status ls_linear_cross_entropy_bw(void *dx, void *dw, const void *x, const void *w,
                                     const int32_t *target, const float *lse, const float *dloss,
                                     int64_t rows, int64_t hidden, int64_t vocab, void *workspace,
                                     size_t workspace_bytes, ls_dtype dt, void *stream);

/* Static, human-readable name of a status code (never NULL). */
const char *ls_status_string(ls_status s);

#ifdef __cplusplus
}
#endif

#endif /* LS_REDUCE_H */
