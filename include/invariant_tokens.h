/*
 * invariant_tokens.h -- C ABI of the token operators: log-probabilities of
 * several given tokens a row with the row's entropy and its most probable
 * tokens, from logits or through the LM head (bf16, or 8-bit rows with
 * scales), their gradients, and the root-mean-square norm that makes the
 * head's input rows.
 *
 * The conventions of invariant_logp.h hold: device pointers owned by the
 * caller, no allocation, work enqueued on `hip_stream` (of the current
 * device), every argument checked on the host before any HIP call, a
 * logp_status code returned, every output element written.  No entry point
 * synchronises, so each can be captured into a HIP graph; a workspace belongs
 * to one call at a time (two streams, or two captured graphs whose replays
 * overlap, need one each).
 *
 * Rows, given tokens and alternatives.  A row has m >= 0 given tokens.  An
 * entry equal to ignore_index is left out: its logp is +0 and it takes no part
 * in a gradient.  A row with m > 0 whose entries are all left out is a padding
 * row: it is not read, its outputs are +0 (ids -1) and its gradients 0.  Any
 * other entry outside [0, v) is invalid: its logp is NaN, nothing out of
 * bounds is read, and in a gradient it matches no column (its g still lowers
 * every probability).  The same token may be given several times.
 * The top_k alternatives of a row are its most probable tokens, greatest logit
 * first, the lowest index first among equals; a NaN logit ranks as -inf (the
 * row's lse, and with it every log-probability, is then NaN).
 *
 * A log-probability is the difference of a logit and the row's fp32 lse, as in
 * logp_fwd, and has the resolution of that lse: 2^-24 of its magnitude.  Where a
 * row's greatest logit is itself a mask (the type's lowest value in every
 * column), log v is lost beside it, in logp and in the gradient (not in the
 * entropy).
 *
 * Batch invariance: a row's outputs depend only on that row (and the weight),
 * not on n, its position, the launch geometry or top_k; lse and entropy have
 * the bits of logp_fwd at the same tile_width, or of linear_logp_fwd.
 */
#ifndef INVARIANT_TOKENS_H
#define INVARIANT_TOKENS_H

#include "invariant_logp.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LOGP_MAX_TOKENS 256 /* given tokens a row */
#define LOGP_MAX_TOP 64     /* alternatives a row */

/*
 * Workspace of token_logp_fwd in bytes: the tile statistics [n, T] and, for
 * top_k > 0, the maxima of the row's groups of 128 columns (64 for LOGP_F32).
 * 0 for arguments token_logp_fwd would reject.
 */
size_t token_logp_fwd_workspace_bytes(int64_t n, int64_t v, int32_t dtype, int32_t tile_width,
                                      int32_t top_k);

/*
 *   logits, dtype, n, v, ld, tile_width: as logp_fwd (rows of any alignment).
 *   tokens        [n, m] of token_dtype (LOGP_I64 or LOGP_I32), contiguous;
 *                 may be NULL when m = 0.  0 <= m <= LOGP_MAX_TOKENS
 *                 (LOGP_ERR_SHAPE).
 *   top_k         0 .. LOGP_MAX_TOP, at most v (LOGP_ERR_VALUE).  v below
 *                 2^32 - 1 when top_k > 0 (LOGP_ERR_SHAPE).
 *   logp_out      fp32 [n, m], may be NULL when m = 0.
 *   lse_out       fp32 [n] or NULL.
 *   entropy_out   fp32 [n] or NULL.
 *   top_logp_out, top_ids_out
 *                 fp32 and int64 [n, top_k], may be NULL when top_k = 0.
 *   workspace     token_logp_fwd_workspace_bytes(...) bytes, 256-byte aligned.
 */
int32_t token_logp_fwd(const void* logits, int32_t dtype, int64_t n, int64_t v, int64_t ld,
                       const void* tokens, int32_t token_dtype, int64_t m, int64_t ignore_index,
                       int32_t tile_width, int32_t top_k, float* logp_out, float* lse_out,
                       float* entropy_out, float* top_logp_out, int64_t* top_ids_out,
                       void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * Gradient of token_logp_fwd's outputs with respect to the logits:
 *   dlogits[r, j] = RNE_dtype(sum of the gradients of r's entries at j
 *                             - G[r] p [- gH[r] p (x - lse[r] + H[r])]),
 *   p = exp(x - lse[r]),  G[r] = the sum of all of r's entry gradients.
 *   tokens, m, ignore_index: the forward's.
 *   top_ids, top_k: the forward's alternatives (negative ids, as padding
 *                 rows have, are left out); NULL and 0 when no gradient comes
 *                 in for them.
 *   lse           fp32 [n] of the forward.
 *   grad_logp     fp32 [n, m] (NULL only when m = 0).
 *   grad_top_logp fp32 [n, top_k] (NULL only when top_k = 0).
 *   entropy, grad_entropy: fp32 [n] each, both NULL or both set.
 *   dlogits_out   [n, ld_out] of the logits dtype, may be exactly the logits
 *                 buffer (in place).  Padding rows are written +0.
 */
int32_t token_logp_bwd(const void* logits, int32_t dtype, int64_t n, int64_t v, int64_t ld,
                       const void* tokens, int32_t token_dtype, int64_t m, int64_t ignore_index,
                       const int64_t* top_ids, int32_t top_k, const float* lse,
                       const float* grad_logp, const float* grad_top_logp, const float* entropy,
                       const float* grad_entropy, void* dlogits_out, int64_t ld_out,
                       void* hip_stream);

/* Options of a linear_token_logp_fwd call, for its workspace size. */
enum logp_token_flags {
  LOGP_TOKEN_KEEPS_LOGITS = 1, /* logits_out is given */
  LOGP_TOKEN_ROUND_BF16 = 2,   /* logits_rounding is LOGP_ROUND_BF16 */
  LOGP_TOKEN_Q8 = 4            /* linear_token_logp_q8_fwd */
};

/*
 * Workspace of linear_token_logp_fwd / linear_token_logp_q8_fwd in bytes.
 * The head's rows are taken row_chunk at a time (rounded up to a multiple of
 * 256); per chunk it holds the tile statistics, a re-laid copy of the hidden
 * rows and, unless logits_out is given or the call has no alternatives and at
 * most one given token a row, the chunk's logits (fp32, bf16 with
 * LOGP_TOKEN_ROUND_BF16), 2.5 GB for 4096 rows of 151936 columns.  row_chunk 0
 * takes 4096 rows where the chunk's logits are in the workspace, else 65536.
 * Any row_chunk gives the same bits.  0 for arguments the call would reject.
 */
size_t linear_token_logp_fwd_workspace_bytes(int64_t n, int64_t h, int64_t v, int64_t m,
                                             int32_t top_k, int32_t flags, int64_t row_chunk);

/*
 * token_logp_fwd through the LM head: logits = hidden weight^T, scaled by
 * fl32(1 / temperature), on the products and tile statistics of
 * linear_logp_fwd (the same bits).
 *   hidden, ld_h, weight, ld_w, n, h, v, temperature, logits_rounding,
 *   prepared, prepared_bytes: as linear_logp_fwd.
 *   logits_out    [n, ld_logits] (ld_logits >= v) receiving the unscaled
 *                 logits for linear_token_logp_bwd, or NULL.  logits_dtype
 *                 LOGP_F32, or LOGP_BF16 only with LOGP_ROUND_BF16.
 *   the rest: as token_logp_fwd.  v at most 2^31.
 */
int32_t linear_token_logp_fwd(const void* hidden, int64_t ld_h, const void* weight, int64_t ld_w,
                              int64_t n, int64_t h, int64_t v, const void* tokens,
                              int32_t token_dtype, int64_t m, int64_t ignore_index,
                              float temperature, int32_t logits_rounding, int32_t top_k,
                              float* logp_out, float* lse_out, float* entropy_out,
                              float* top_logp_out, int64_t* top_ids_out, void* logits_out,
                              int32_t logits_dtype, int64_t ld_logits, const void* prepared,
                              size_t prepared_bytes, int64_t row_chunk, void* workspace,
                              size_t workspace_bytes, void* hip_stream);

/*
 * Workspace of linear_token_logp_bwd in bytes for the same flags
 * (logp_bwd_flags) and vocab_chunk.
 */
size_t linear_token_logp_bwd_workspace_bytes(int64_t n, int64_t h, int64_t v, int32_t flags,
                                             int64_t vocab_chunk);

/*
 * Backward of linear_token_logp_fwd: linear_logp_bwd with a list of entries a
 * row.  dz is rounded to bf16 once, after the entries' gradients are added.
 * dhidden is the sum, in ascending order, of the fp32 sums over segments of the
 * vocabulary (v / 4 columns, rounded up to a multiple of 1024, at least 4096 and
 * at most 16384); vocab_chunk (0 = the library's default) is rounded up to whole
 * segments, and any value gives the same bits.
 *   logp, top_logp: the forward's outputs ([n, m], [n, top_k]).
 *   the rest: as linear_logp_bwd and token_logp_bwd.
 */
int32_t linear_token_logp_bwd(const void* hidden, int64_t ld_h, const void* weight, int64_t ld_w,
                              int64_t n, int64_t h, int64_t v, const void* tokens,
                              int32_t token_dtype, int64_t m, int64_t ignore_index,
                              const int64_t* top_ids, int32_t top_k, float temperature,
                              int32_t logits_rounding, const void* saved_logits,
                              int32_t saved_dtype, int64_t ld_saved, const void* prepared,
                              size_t prepared_bytes, const float* lse, const float* logp,
                              const float* top_logp, const float* grad_logp,
                              const float* grad_top_logp, const float* entropy,
                              const float* grad_entropy, int32_t out_dtype, void* dhidden,
                              int64_t ld_dh, void* dweight, int64_t ld_dw, int64_t vocab_chunk,
                              void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * The forward through an 8-bit LM head (frozen weights: scoring, decoding):
 *   logits[r, j] = (sum_k hidden[r, k] weight[j, k]) hidden_scale[r] weight_scale[j]
 * with hidden [n, ld_h] and weight [v, ld_w] in e4m3 (OCP 8-bit floating
 * point: 4 exponent bits, 3 mantissa bits, largest value 448), exact products
 * and fp32 sums, no split.  h a multiple of 64; 16-byte aligned rows at most
 * 2^23 bytes apart (LOGP_ERR_SHAPE); scales fp32 [n] and [v].  The rest: as
 * linear_token_logp_fwd (workspace flag LOGP_TOKEN_Q8); its own arithmetic, so
 * its bits are not linear_token_logp_fwd's, but they are batch invariant too.
 */
int32_t linear_token_logp_q8_fwd(const void* hidden, int64_t ld_h, const float* hidden_scale,
                                 const void* weight, int64_t ld_w, const float* weight_scale,
                                 int64_t n, int64_t h, int64_t v, const void* tokens,
                                 int32_t token_dtype, int64_t m, int64_t ignore_index,
                                 float temperature, int32_t top_k, float* logp_out,
                                 float* lse_out, float* entropy_out, float* top_logp_out,
                                 int64_t* top_ids_out, int64_t row_chunk, void* workspace,
                                 size_t workspace_bytes, void* hip_stream);

/*
 * Root-mean-square norm with the residual's addition:
 *   s = RNE_dtype(x + residual)            (x itself without a residual)
 *   y = RNE_dtype(s * rstd * weight),  rstd = 1 / sqrt(mean(s^2) + eps)
 * The stored s is what is normed, so the fused call has the bits of an
 * addition followed by the norm of its stored result.  Sums in fp32 through a
 * tree fixed by h alone; squares past fp32's range (values of about 1e19) give
 * rstd 0, and squares below it count as 0.
 *   x [n, ld_x], residual [n, ld_r] (NULL: none), weight [h], y [n, ld_y],
 *   sum_out [n, ld_s] (NULL only without a residual): dtype LOGP_F32, LOGP_BF16
 *   or LOGP_F16; any alignment, whole 16-byte accesses where the rows are
 *   16-byte aligned.  sum_out may be exactly x or residual (in place), y may
 *   be exactly x when sum_out is another buffer or absent.
 *   1 <= h <= 65536 (LOGP_ERR_SHAPE); eps finite and >= 0 (LOGP_ERR_VALUE).
 *   rstd_out  fp32 [n] or NULL (the backward's input).
 */
int32_t rms_norm_fwd(const void* x, int64_t ld_x, const void* residual, int64_t ld_r,
                     const void* weight, int32_t dtype, int64_t n, int64_t h, float eps, void* y,
                     int64_t ld_y, void* sum_out, int64_t ld_s, float* rstd_out,
                     void* hip_stream);

/*
 * rms_norm_fwd with 8-bit rows as output:
 *   t = s * rstd * weight (fp32),  a = max(max|t|, 448 * 2^-126),
 *   scale[r] = a / 448,  q = RNE_e4m3(t * (448 / a))
 *                                          (a row of zeros: scale 0, q 0)
 * q_out [n, ld_q] bytes, scale_out fp32 [n].  A row with an infinity or a NaN
 * gives NaN.  weight NULL: no norm, t = s (8-bit rows of a weight matrix).
 */
int32_t rms_norm_q8_fwd(const void* x, int64_t ld_x, const void* residual, int64_t ld_r,
                        const void* weight, int32_t dtype, int64_t n, int64_t h, float eps,
                        void* q_out, int64_t ld_q, float* scale_out, void* sum_out, int64_t ld_s,
                        void* hip_stream);

/*
 * Workspace of rms_norm_bwd in bytes: the weight gradient's partial sums.
 */
size_t rms_norm_bwd_workspace_bytes(int64_t n, int64_t h);

/*
 * Gradient of rms_norm_fwd, given those of y (dy) and of s (ds, or NULL):
 *   u = s rstd,  dx = RNE_dtype(ds + rstd (dy w - u mean(dy w u)))
 *   dweight = RNE_dtype(sum_r dy u)        (rows summed in a fixed order)
 * dx is the gradient of x and of the residual alike.
 *   s [n, ld_s]: the forward's stored sum (x without a residual); rstd fp32
 *   [n]; dx [n, ld_dx], may be exactly dy or ds; dweight [h] of dtype, or NULL
 *   (then no workspace is needed).  n = 0 writes dweight with zeros.
 */
int32_t rms_norm_bwd(const void* s, int64_t ld_s, const void* weight, const float* rstd,
                     const void* dy, int64_t ld_dy, const void* ds, int64_t ld_ds, int32_t dtype,
                     int64_t n, int64_t h, void* dx, int64_t ld_dx, void* dweight,
                     void* workspace, size_t workspace_bytes, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* INVARIANT_TOKENS_H */
