/*
 * invariant_layers.h -- C ABI of the operators at the other end of the tied
 * table and around the residual stream: the embedding with its gradient,
 * dropout, the layer norm with its gradient, and rows in 4 bits.
 *
 * The conventions of invariant_logp.h hold: device pointers owned by the
 * caller, no allocation, work enqueued on `hip_stream` (of the current
 * device), every argument checked on the host before any HIP call, a
 * logp_status code returned, every output element written.  No entry point
 * synchronises, so each can be captured into a HIP graph; a workspace belongs
 * to one call at a time.
 *
 * Batch invariance: a row's outputs depend only on that row (and the
 * parameters), not on n, its position or the launch geometry.  Dropout's mask
 * is a function of the seed, the draw, the row's number and the column, and a
 * row of the embedding's gradient one of its token's own occurrences, in order.
 */
#ifndef INVARIANT_LAYERS_H
#define INVARIANT_LAYERS_H

#include "invariant_logp.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Rows of a table by token, times a scale:
 *   out[i] = RNE_dtype(scale * table[tokens[i]])
 *   table  [v, ld_t] and out [n, ld_o] of dtype LOGP_F32, LOGP_BF16 or LOGP_F16,
 *          any alignment, whole 16-byte accesses where the rows are 16-byte
 *          aligned.  h at most 2^24 (LOGP_ERR_SHAPE), scale finite
 *          (LOGP_ERR_VALUE).
 *   tokens [n] of token_dtype (LOGP_I64 or LOGP_I32).  A token equal to
 *          ignore_index gives a row of +0; any other outside [0, v) is
 *          invalid: its row is NaN and nothing out of bounds is read.
 */
int32_t embedding_fwd(const void* table, int64_t ld_t, int64_t v, int64_t h, int32_t dtype,
                      const void* tokens, int32_t token_dtype, int64_t n, int64_t ignore_index,
                      float scale, void* out, int64_t ld_o, void* hip_stream);

/*
 * The same from 4-bit rows (fp4_quantize): data [v, ld_d] and scales [v, ld_s]
 * bytes, out of out_dtype.  h a multiple of 32; 16-byte aligned data rows
 * (LOGP_ERR_ALIGN).  Table values are those of fp32: exact, or an infinity where
 * scale bytes 253 and 254 pass its range.
 */
int32_t embedding_fp4_fwd(const void* data, int64_t ld_d, const void* scales, int64_t ld_s,
                          int64_t v, int64_t h, const void* tokens, int32_t token_dtype, int64_t n,
                          int64_t ignore_index, float scale, int32_t out_dtype, void* out,
                          int64_t ld_o, void* hip_stream);

/*
 * Workspace of embedding_bwd in bytes: the sorted tokens and the partial rows of
 * tokens that occur more than 32 times.  0 for arguments embedding_bwd would
 * reject.
 */
size_t embedding_bwd_workspace_bytes(int64_t n, int64_t v, int64_t h);

/*
 * Gradient of embedding_fwd with respect to the table, by sorted tokens:
 *   dtable[t] = RNE([dtable[t] +] scale * sum of dy[i] over i with tokens[i] = t)
 * in fp32, occurrences in ascending i: chains of 32, and where there are several
 * of them eight chains of every eighth, then those in order.  Entries equal to
 * ignore_index and invalid ones are left out (their dy is not read).
 *   dy     [n, ld_y] of dtype; n at most 2^24, v at most 2^31 (LOGP_ERR_SHAPE).
 *   dtable [v, ld_t] of out_dtype: LOGP_F32 or dtype (LOGP_ERR_DTYPE).
 *   accumulate 0: every row is written (+0 for absent tokens); 1: the sums are
 *          added to what is there (the gradient of a tied LM head, say) and
 *          the rows of absent tokens stay as they are.
 */
int32_t embedding_bwd(const void* dy, int64_t ld_y, int32_t dtype, const void* tokens,
                      int32_t token_dtype, int64_t n, int64_t v, int64_t h, int64_t ignore_index,
                      float scale, int32_t out_dtype, int32_t accumulate, void* dtable,
                      int64_t ld_t, void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * Dropout with the residual's addition:
 *   out[r, j] = RNE_dtype(residual[r, j] + (u >= T ? x[r, j] * c : 0))
 * T = floor(65536 p + 1/2), c = 65536 / (65536 - T) as fp32 (all is dropped
 * where T = 65536).  u is one of the eight 16-bit numbers that Philox-4x32-10
 * gives for the key seed (low word, high word) and the counter
 *   (j / 8, R mod 2^32, R / 2^32, draw),  R = first_row + r:
 * number j mod 8, two a word, the low half first.  A dropped element does not
 * take part, whatever it is.  The gradient of x is the same call on the gradient
 * of out without a residual; that of the residual is the gradient of out.
 *   x [n, ld_x], residual [n, ld_r] (NULL: none), out [n, ld_o] of dtype;
 *   out may be exactly x or residual.  h at most 2^24 (LOGP_ERR_SHAPE).
 *   p in [0, 1], draw in [0, 2^32), first_row from 0 to 2^63 - 2^31
 *   (LOGP_ERR_VALUE).
 *   seed_at NULL, or the seed's address on the device, which is read in place of
 *   `seed` when the kernel runs (a captured graph draws anew as it changes).
 */
int32_t dropout_fwd(const void* x, int64_t ld_x, const void* residual, int64_t ld_r, int32_t dtype,
                    int64_t n, int64_t h, double p, int64_t seed, const int64_t* seed_at,
                    int64_t draw, int64_t first_row, void* out, int64_t ld_o, void* hip_stream);

/*
 * Layer norm with dropout and the residual's addition:
 *   s = RNE_dtype(residual + dropped(x))       (dropout_fwd; x itself without)
 *   y = RNE_dtype((s - m) * rstd * weight + bias)
 *   m = mean(s), rstd = 1 / sqrt(mean((s - m)^2) + eps)
 * The stored s is what is normed, so the fused call has the bits of dropout_fwd
 * followed by the norm of its output.  Sums in fp32 through a tree fixed by h
 * alone; squares past fp32's range (differences from the mean of about 1e19)
 * give rstd 0, a sum past it a row of NaN.
 *   x [n, ld_x], residual [n, ld_r] (NULL: none), weight [h], bias [h] (NULL:
 *   none), y [n, ld_y], sum_out [n, ld_s] (NULL only where s is x): dtype, any
 *   alignment.  sum_out may be exactly x or residual, y exactly x when sum_out
 *   is another buffer or absent.  1 <= h <= 65536 (LOGP_ERR_SHAPE); eps finite
 *   and >= 0 (LOGP_ERR_VALUE).
 *   p, seed, seed_at, draw, first_row: as dropout_fwd; p 0: no dropout.
 *   mean_out, rstd_out  fp32 [n], or NULL (the backward's inputs).
 */
int32_t layer_norm_fwd(const void* x, int64_t ld_x, const void* residual, int64_t ld_r,
                       const void* weight, const void* bias, int32_t dtype, int64_t n, int64_t h,
                       float eps, double p, int64_t seed, const int64_t* seed_at, int64_t draw,
                       int64_t first_row, void* y, int64_t ld_y, void* sum_out, int64_t ld_s,
                       float* mean_out, float* rstd_out, void* hip_stream);

/*
 * Workspace of layer_norm_bwd in bytes: the partial sums of dweight and dbias.
 */
size_t layer_norm_bwd_workspace_bytes(int64_t n, int64_t h);

/*
 * Gradient of layer_norm_fwd, given those of y (dy) and of s (ds, or NULL):
 *   u = (s - m) rstd, g = dy weight
 *   d = ds + rstd (g - mean(g) - u mean(g u))
 *   p 0:  dx = RNE_dtype(d), the gradient of x and of the residual alike;
 *   else: dresidual = RNE_dtype(d), dx = RNE_dtype(u' >= T ? d * c : 0) with the
 *         forward's numbers u'
 *   dweight = RNE_dtype(sum_r dy u), dbias = RNE_dtype(sum_r dy), rows summed in
 *   a fixed order
 *   s [n, ld_s]: the forward's stored sum; mean, rstd fp32 [n]; dx [n, ld_dx] and
 *   dresidual [n, ld_dr] (NULL: not asked for; NULL for p 0, LOGP_ERR_VALUE)
 *   each may be exactly dy or ds, not one another.  dweight, dbias [h] of
 *   dtype, or NULL (with both NULL no workspace is needed).  n = 0 writes them
 *   with zeros.
 */
int32_t layer_norm_bwd(const void* s, int64_t ld_s, const void* weight, const float* mean,
                       const float* rstd, const void* dy, int64_t ld_dy, const void* ds,
                       int64_t ld_ds, int32_t dtype, int64_t n, int64_t h, double p, int64_t seed,
                       const int64_t* seed_at, int64_t draw, int64_t first_row, void* dx,
                       int64_t ld_dx, void* dresidual, int64_t ld_dr, void* dweight, void* dbias,
                       void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * 4-bit rows of x [n, ld_x] (dtype): two e2m1 values a byte, the even column in
 * the low half, and one scale byte b for every 32 columns, which stands for
 * 2^(b - 127) (255: NaN).  e2m1 codes 0 to 7 stand for 0, 1/2, 1, 3/2, 2, 3, 4, 6,
 * codes 8 to 15 for their negatives.  b is the smallest from 1 to 252 that
 * brings the group's magnitudes within 6 (past 252 they saturate), 255 where the
 * group holds an infinity or a NaN; values are rounded to the nearest, ties to
 * an even code.
 *   data [n, ld_d] and scales [n, ld_s] bytes.  h a multiple of 32, at most 2^24
 *   (LOGP_ERR_SHAPE); 16-byte aligned data rows (LOGP_ERR_ALIGN).
 */
int32_t fp4_quantize(const void* x, int64_t ld_x, int32_t dtype, int64_t n, int64_t h, void* data,
                     int64_t ld_d, void* scales, int64_t ld_s, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* INVARIANT_LAYERS_H */
