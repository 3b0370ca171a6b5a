/*
 * lrs_lm.h -- operators of recurrent language models in liblrs.so: a gated
 * linear recurrence with a learned decay (forward, backward, single tokens), a
 * layer norm with the residual added in (forward, backward), and the softmax
 * cross entropy of a linear head over a large vocabulary, with its gradient,
 * without storing all of its logits.
 *
 * The conventions of lrs.h hold: device pointers owned by the caller, a
 * caller's workspace sized by a query, an opaque stream, error codes and no
 * exceptions, arguments validated before any launch, element type LRS_F32 or
 * LRS_BF16 with fp32 state, statistics, parameters and arithmetic (the products
 * of the cross entropy take 16-bit factors, as described there), and results
 * that are bitwise the same from call to call.  Outputs must not overlap
 * inputs or other outputs unless a function says so.
 */
#ifndef LRS_LM_H
#define LRS_LM_H

#include "lrs.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------- gated linear recurrence --- */

/* For every step t, sequence b and feature d, with pre-activations z_r, z_i
 * and the input x (the three parts of a projection made outside):
 *   r = sigmoid(z_r + bias_r),  i = sigmoid(z_i + bias_i),
 *   a = exp(-c softplus(decay) r),  m = sqrt(1 - a^2),
 *   h_t = a h_{t-1} + m i x;
 * where reset[t,b] != 0 a new document starts: a = 0 and m = 1, so that nothing
 * of the state before reaches h_t (nor a gradient back), NaN and infinities
 * included.
 * z_r, z_i, x : [T,B,D], element (t,b,d) at (t*B + b)*ld + d, ld >= D, so that
 *               slices of one [T,B,3D] projection need no copy.
 * bias_r, bias_i, decay : [D] fp32.  reset: [T,B] bytes, or NULL for none.
 * h0          : [B,D] fp32, or NULL (zero).
 * h           : [T,B,D] contiguous output.  h_last: [B,D] fp32 output or NULL.
 * checkpoints : fp32 output [lrs_glr_checkpoint_rows(T), B, D], the states that
 *               enter each stretch of time steps, which lrs_glr_bwd reads (it
 *               recomputes the states between them); or NULL.
 * c           : positive and finite.
 * Supported while B*D stays below 2^31 and B*ld below 2^30. */
LRS_API int64_t lrs_glr_checkpoint_rows(int64_t T);
LRS_API size_t lrs_glr_workspace_bytes(int64_t T, int64_t B, int64_t D);
LRS_API int lrs_glr_fwd(const void *z_r, const void *z_i, const void *x, int64_t ld,
                        const float *bias_r, const float *bias_i, const float *decay,
                        const uint8_t *reset, const float *h0, void *h, float *h_last,
                        float *checkpoints, int64_t T, int64_t B, int64_t D, float c,
                        int io_dtype, void *workspace, size_t workspace_bytes, void *stream);

/* Its backward pass.  With lam_t the whole gradient of h_t,
 *   lam_t = grad_h_t + a_{t+1} lam_{t+1}   (lam_T adds grad_h_last):
 *   dx = lam m i,  dz_i = lam m x i (1 - i),
 *   dla = lam (a h_{t-1} - (a^2 / m) i x)  (0 at a reset, and with it dz_r, whatever
 *                                          z_r is there),
 *   dz_r = dla la (1 - r),  ddecay = sum dla (-c sigmoid(decay)) r,
 *   dbias_r, dbias_i = sums of dz_r, dz_i over steps and sequences,  dh0 = a_1 lam_1.
 * The term with 1/m is 0 where m is 0 (a gate closed to the last bit).
 * checkpoints : as lrs_glr_fwd wrote them for the same inputs.
 * grad_h      : [T,B,D] contiguous, I/O type.  grad_h_last: [B,D] fp32 or NULL.
 * grad_zr, grad_zi, grad_x : I/O type, rows ld_grad apart (slices of one
 *               [T,B,3D] gradient may interleave).
 * grad_bias_r, grad_bias_i, grad_decay : [D] fp32.  grad_h0: [B,D] fp32 or NULL. */
LRS_API size_t lrs_glr_bwd_workspace_bytes(int64_t T, int64_t B, int64_t D);
LRS_API int lrs_glr_bwd(const void *z_r, const void *z_i, const void *x, int64_t ld,
                        const float *bias_r, const float *bias_i, const float *decay,
                        const uint8_t *reset, const float *checkpoints, const void *grad_h,
                        const float *grad_h_last, void *grad_zr, void *grad_zi, void *grad_x,
                        int64_t ld_grad, float *grad_bias_r, float *grad_bias_i,
                        float *grad_decay, float *grad_h0, int64_t T, int64_t B, int64_t D,
                        float c, int io_dtype, void *workspace, size_t workspace_bytes,
                        void *stream);

/* One token for each of B sequences.  state: [S,D] fp32, updated in place.
 * slots: [B] int32, the row of `state` that each sequence owns; a sequence
 * whose slot is outside [0, S) is idle: its h is 0 and no state changes.  Slots
 * in use must differ from each other.  NULL: sequence b owns row b (S >= B).
 * z_r, z_i, x: [B,D], rows ld apart.  h: [B,D] contiguous. */
LRS_API int lrs_glr_step(const void *z_r, const void *z_i, const void *x, int64_t ld,
                         const float *bias_r, const float *bias_i, const float *decay,
                         const int32_t *slots, float *state, void *h, int64_t B, int64_t D,
                         int64_t S, float c, int io_dtype, void *stream);

/* ---------------------------------------------------------- layer norm --- */

/* Layer norm over the last axis of [R,D] rows, with the residual added first:
 *   s = x + residual (rounded to the I/O type; s = x without a residual),
 *   y = (s - mean) rstd gamma + beta,  rstd = 1 / sqrt(var + eps),
 * with the variance taken about the mean over D.
 * x, residual, y, sum : [R,D], I/O type.  residual may be NULL; sum receives s
 *   and is required with a residual (it may be x's or the residual's own
 *   buffer: the residual stream in place), and NULL without.
 * gamma, beta : [D] fp32; beta may be NULL (zero).
 * mean, rstd  : [R] fp32 outputs (both or neither), as lrs_layernorm_bwd takes
 *   them.  eps >= 0 and finite.
 * Supported while R stays below 2^22, or below 2^26 - 4 where D <= 1024. */
LRS_API int lrs_layernorm_fwd(const void *x, const void *residual, const float *gamma,
                              const float *beta, void *y, void *sum, float *mean, float *rstd,
                              int64_t R, int64_t D, float eps, int io_dtype, void *stream);

/* Its backward pass.  With q = grad_y gamma and xh = (s - mean) rstd,
 *   dx = rstd (q - mean(q) - xh mean(q xh)) + grad_sum,
 *   dgamma = sum over rows of grad_y xh,  dbeta = sum over rows of grad_y.
 * s        : what was normalised (x, or lrs_layernorm_fwd's sum).
 * grad_sum : gradient that reaches s from elsewhere (the residual stream), or
 *            NULL.  grad_x: gradient of x and of the residual; it may be
 *            grad_y's or grad_sum's own buffer.
 * grad_gamma, grad_beta : [D] fp32 (grad_beta may be NULL). */
LRS_API size_t lrs_layernorm_bwd_workspace_bytes(int64_t R, int64_t D);
LRS_API int lrs_layernorm_bwd(const void *s, const float *gamma, const float *mean,
                              const float *rstd, const void *grad_y, const void *grad_sum,
                              void *grad_x, float *grad_gamma, float *grad_beta, int64_t R,
                              int64_t D, int io_dtype, void *workspace, size_t workspace_bytes,
                              void *stream);

/* ------------------------------- cross entropy of a linear head --- */

/* Softmax cross entropy of the logits l = x w^T against one class a row:
 *   lse_n = log sum_v exp l_nv,   loss_n = lse_n - l_{n,target_n}.
 * A row whose target lies outside [0, V) is ignored: loss 0, no gradient, and
 * its x reaches no gradient of w (lse is written all the same).  The logits are
 * made tile by tile on the matrix cores: the forward stores none, the gradient
 * the exponentials of a piece of the rows at a time (below).
 * x: [N,D], w: [V,D], I/O type.  target: [N] int64.  loss, lse: [N] fp32.
 * fp32 operands are split into two scaled fp16 parts and multiplied in three
 * products.  A sum of products is then off by up to 2^-21 of the sum of its
 * absolute terms (not of the result, which may cancel), and a value below 2^-17
 * of the largest it is scaled with is known to 2^-39 of that: the largest of its
 * row for the logits, of the whole array for the gradients.  An infinity in an
 * fp32 operand counts as NaN.
 * Supported while N, V and D stay below 2^21.
 * The workspace query takes whether the call makes the gradient. */
LRS_API size_t lrs_linear_ce_workspace_bytes(int64_t N, int64_t V, int64_t D, int io_dtype,
                                             int backward);
LRS_API int lrs_linear_ce_fwd(const void *x, const void *w, const int64_t *target, float *loss,
                              float *lse, int64_t N, int64_t V, int64_t D, int io_dtype,
                              void *workspace, size_t workspace_bytes, void *stream);

/* Its gradient for given dL/dloss: with G = (exp(l - lse) - onehot) grad_loss
 * (rows of 0 where ignored), grad_x = G w and grad_w = G^T x, I/O type.  The
 * rows are taken in pieces of at least 256 rows: the exponentials of a piece's
 * logits (made again here) and its G are kept in the workspace, 1 GiB for bf16
 * and 2 GiB for fp32 at most unless 256 rows take more.  G is rounded to bf16
 * for bf16 inputs, from exponentials kept in fp16: a class more than 20 nats
 * below the likeliest of the 32 to 128 classes next to it begins to lose
 * digits in that row's gradient, and has none from 27 nats on.
 * For fp32 inputs G is known to 2^-22 of itself or to 2^-50.
 * lse: as lrs_linear_ce_fwd wrote it.  grad_loss: [N] fp32. */
LRS_API int lrs_linear_ce_bwd(const void *x, const void *w, const int64_t *target,
                              const float *lse, const float *grad_loss, void *grad_x,
                              void *grad_w, int64_t N, int64_t V, int64_t D, int io_dtype,
                              void *workspace, size_t workspace_bytes, void *stream);

/* Both in one call, for a grad_loss that is known before the loss is (a mean
 * over the rows that count): the results of lrs_linear_ce_fwd and then
 * lrs_linear_ce_bwd, with the logits made once instead of twice. */
LRS_API int lrs_linear_ce_fwd_bwd(const void *x, const void *w, const int64_t *target,
                                  const float *grad_loss, float *loss, float *lse, void *grad_x,
                                  void *grad_w, int64_t N, int64_t V, int64_t D, int io_dtype,
                                  void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LRS_LM_H */
