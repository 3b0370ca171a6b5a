/*
 * lrs_block.h -- operators of a delta-rule language model in liblrs.so, beside
 * those of lrs_lm.h: the gated delta rule (forward, backward, single tokens),
 * a root-mean-square norm with the residual added in (forward, backward, and an
 * output in 8 bits with scales), and the log probabilities of given tokens with
 * the entropy and the likeliest alternatives (forward, backward).
 *
 * The conventions of lrs.h hold: device pointers owned by the caller, a
 * caller's workspace sized by a query, an opaque stream, error codes and no
 * exceptions, arguments validated before any launch, element type LRS_F32 or
 * LRS_BF16 with fp32 state, statistics, parameters and arithmetic (the products
 * of the delta rule take 16-bit factors, as described there), and results
 * that are bitwise the same from call to call.  Outputs must not overlap
 * inputs or other outputs unless a function says so.
 */
#ifndef LRS_BLOCK_H
#define LRS_BLOCK_H

#include "lrs.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------- gated delta rule --- */

/* For every sequence b and head h a [K,V] state S, from state0, and for every
 * step t, with a = exp(log_decay_t) (S = 0 instead of a S where reset[t,b] != 0:
 * a new document starts, and nothing of the state before reaches it, nor a
 * gradient back, NaN and infinities included):
 *   S <- a S,  u = beta_t (v_t - S^T k_t),  S <- S + k_t u^T,
 *   o_t = scale S^T q_t.
 * H heads of v, log_decay, beta and o share Hk heads of q and k (H a multiple
 * of Hk): head h reads q and k of head h / (H / Hk).
 * q, k   : [T,B,Hk,K], element (t,b,hk,i) at (t*B + b)*ld + hk*K + i, ld >= Hk*K,
 *          so that slices of one projection need no copy; v: [T,B,H,V], rows
 *          ld_v apart.  A k of length 1 and a beta in [0,2] keep the state from
 *          growing; neither is asked for.
 * log_decay, beta : [T,B,H] fp32 contiguous (a log_decay under -16384 counts as
 *          -16384: exp of it is 0 either way).  A log_decay may be above 0, but where its
 *          sum over neighbouring steps of a chunk of 64 passes 88 their exp is infinite,
 *          and gives NaN also for a state of 0.
 * reset  : [T,B] bytes, or NULL for none; each document in a chunk of 64 steps costs the
 *          chunk's work again.  state0: [B,H,K,V] fp32, or NULL (zero).
 * o      : [T,B,H,V] contiguous output.  state: [B,H,K,V] fp32 output, the state
 *          after the last step, or NULL; it may be state0's own buffer.
 * checkpoints : fp32 output [lrs_gdr_checkpoint_rows(T), B, H, K + 64, V'], V' = V
 *          rounded up to a multiple of 4, for each chunk of 64 steps the state that
 *          enters it and v - S^T k of its steps, which lrs_gdr_bwd reads; or NULL.
 *          Its padding needs no values.
 * Products take factors of two fp16 parts, scaled by a power of two (one part
 * where bf16 inputs need no more): a factor is known to 2^-22 of itself or to
 * 2^-39 of the largest of its row or column, whichever is more.  A value that is
 * not finite makes what its document computes from it NaN or infinite, up to
 * 63 steps before it (its chunk) and in the columns of V and heads it reaches.
 * Supported: K <= 128, B*H*V and B*ld below 2^23 for every row pitch ld, (K+64)*V' below 2^29, and
 * the chunks ceil(T/64)*B*H below 2^24 (2^23 for lrs_gdr_bwd), times ceil(V/16) below 2^26. */
LRS_API int64_t lrs_gdr_checkpoint_rows(int64_t T);
LRS_API size_t lrs_gdr_workspace_bytes(int64_t T, int64_t B, int64_t H, int64_t Hk, int64_t K,
                                       int64_t V, int io_dtype);
LRS_API int lrs_gdr_fwd(const void *q, int64_t ld_q, const void *k, int64_t ld_k, const void *v,
                        int64_t ld_v, const float *log_decay, const float *beta,
                        const uint8_t *reset, const float *state0, void *o, float *state,
                        float *checkpoints, int64_t T, int64_t B, int64_t H, int64_t Hk,
                        int64_t K, int64_t V, float scale, int io_dtype, void *workspace,
                        size_t workspace_bytes, void *stream);

/* Its backward pass for the same inputs and the checkpoints that lrs_gdr_fwd
 * wrote for them.
 * grad_o     : [T,B,H,V] contiguous, I/O type.  grad_state: [B,H,K,V] fp32, the
 *              gradient of the last state, or NULL (zero).
 * grad_q, grad_k, grad_v : I/O type, shaped as q, k and v, rows ld_g* apart
 *              (slices of one gradient may interleave); heads that share q and k
 *              are summed in fp32.
 * grad_log_decay (0 at a reset), grad_beta : [T,B,H] fp32.
 * grad_state0 : [B,H,K,V] fp32 or NULL; it may be grad_state's own buffer. */
LRS_API size_t lrs_gdr_bwd_workspace_bytes(int64_t T, int64_t B, int64_t H, int64_t Hk, int64_t K,
                                           int64_t V, int io_dtype);
LRS_API int lrs_gdr_bwd(const void *q, int64_t ld_q, const void *k, int64_t ld_k, const void *v,
                        int64_t ld_v, const float *log_decay, const float *beta,
                        const uint8_t *reset, const float *checkpoints, const void *grad_o,
                        const float *grad_state, void *grad_q, int64_t ld_gq, void *grad_k,
                        int64_t ld_gk, void *grad_v, int64_t ld_gv, float *grad_log_decay,
                        float *grad_beta, float *grad_state0, int64_t T, int64_t B, int64_t H,
                        int64_t Hk, int64_t K, int64_t V, float scale, int io_dtype,
                        void *workspace, size_t workspace_bytes, void *stream);

/* One token for each of B sequences, in fp32 throughout.  state: [S,H,K,V] fp32,
 * updated in place.  slots: [B] int32, the row of `state` that each sequence
 * owns; a sequence whose slot is outside [0, S) is idle: its o is 0 and no state
 * changes.  Slots in use must differ from each other.  NULL: sequence b owns row
 * b (S >= B).  q, k: [B,Hk,K], v: [B,H,V], rows ld_* apart; log_decay, beta:
 * [B,H]; o: [B,H,V] contiguous.
 * Supported: K <= 128, and B*H*ceil(V/128) * 256 below 2^32. */
LRS_API int lrs_gdr_step(const void *q, int64_t ld_q, const void *k, int64_t ld_k, const void *v,
                         int64_t ld_v, const float *log_decay, const float *beta,
                         const int32_t *slots, float *state, void *o, int64_t B, int64_t H,
                         int64_t Hk, int64_t K, int64_t V, int64_t S, float scale, int io_dtype,
                         void *stream);

/* ------------------------------------------- root-mean-square norm --- */

/* Over the last axis of [R,D] rows, with the residual added first:
 *   s = x + residual (rounded to the I/O type; s = x without a residual),
 *   y = s rstd gamma,  rstd = 1 / sqrt(mean(s^2) + eps).
 * x, residual, y, sum : [R,D], I/O type.  residual may be NULL; sum receives s
 *   and is required with a residual (it may be x's or the residual's own
 *   buffer: the residual stream in place), and NULL without.
 * gamma : [D] fp32.  rstd: [R] fp32 output or NULL.  eps >= 0 and finite.
 * Squares are summed in fp32: where they pass its range rstd is 0, and y with it.
 * Supported while R stays below 2^22, or below 2^26 - 4 where D <= 1024. */
LRS_API int lrs_rmsnorm_fwd(const void *x, const void *residual, const float *gamma, void *y,
                            void *sum, float *rstd, int64_t R, int64_t D, float eps, int io_dtype,
                            void *stream);

/* The same with y in 8 bits: for each group of `group` features of a row (128,
 * the last one shorter where D is no multiple; 0: the whole row)
 *   scale = max |y| / 448, at least 2^-120 (1 where every y is 0),
 *   q = y / scale rounded to e4m3 (nearest, ties to even),
 * taken from y in fp32, each quotient rounded to fp32 first.  q: [R,D] bytes, e4m3 without infinities (OCP); scales:
 * [R, ceil(D / group)] fp32.  A group with a NaN or an infinity has a scale that
 * is not finite and q NaN.  Supported as lrs_rmsnorm_fwd. */
LRS_API int lrs_rmsnorm_fwd_fp8(const void *x, const void *residual, const float *gamma,
                                void *q, float *scales, void *sum, int64_t R, int64_t D,
                                int64_t group, float eps, int io_dtype, void *stream);

/* Its backward pass (of lrs_rmsnorm_fwd).  With g = grad_y gamma and xh = s rstd,
 *   dx = rstd (g - xh mean(g xh)) + grad_sum,  dgamma = sum over rows of grad_y xh.
 * s        : what was normalised (x, or lrs_rmsnorm_fwd's sum).
 * grad_sum : gradient that reaches s from elsewhere (the residual stream), or
 *            NULL.  grad_x: gradient of x and of the residual; it may be
 *            grad_y's or grad_sum's own buffer.  grad_gamma: [D] fp32. */
LRS_API size_t lrs_rmsnorm_bwd_workspace_bytes(int64_t R, int64_t D);
LRS_API int lrs_rmsnorm_bwd(const void *s, const float *gamma, const float *rstd,
                            const void *grad_y, const void *grad_sum, void *grad_x,
                            float *grad_gamma, int64_t R, int64_t D, int io_dtype,
                            void *workspace, size_t workspace_bytes, void *stream);

/* ---------------------------------- log probabilities of given tokens --- */

/* From logits l [N,V], rows ld apart:
 *   lse_n = log sum_v exp l_nv,  logprob_n = l_{n,target_n} - lse_n,
 *   entropy_n = -sum_v p_nv log p_nv  (a logit of -infinity adds nothing),
 * and the `top` largest logits of a row, with their log probabilities, in
 * falling order; of equal ones (-0 and +0 are) the lower index comes first, and
 * NaN counts as larger than any number.
 * A target outside [0, V) is ignored: logprob 0 (and no gradient through it).
 * A row with a NaN or +infinity, or with nothing but -infinity, has NaN for its
 * log probabilities and entropy.
 * logits: I/O type.  target: [N] int64.  logprob, entropy, lse: [N] fp32;
 * top_ids: [N,top] int64, top_logprobs: [N,top] fp32 (NULL with top = 0).
 * 0 <= top <= 64 and top <= V.  Supported while N and V stay below 2^24. */
LRS_API int lrs_logprobs_fwd(const void *logits, int64_t ld, const int64_t *target,
                             float *logprob, float *entropy, float *lse, int64_t *top_ids,
                             float *top_logprobs, int64_t N, int64_t V, int64_t top, int io_dtype,
                             void *stream);

/* The gradient of logprob and entropy:
 *   grad_l = grad_logprob (onehot - p) - grad_entropy p (log p + entropy),
 * where a p of 0 adds nothing, and 0 in a row whose target is ignored and whose grad_entropy
 * is 0, whatever its logits are.  lse, entropy: as lrs_logprobs_fwd wrote them.  With lse as it
 * was rounded, p is known to some 2^-24 (|lse| + 3 |log p|) of itself, which is also what
 * onehot - p keeps of a nearly certain target; from |lse| = 256 on the row is summed again
 * instead (one more reading of it).  grad_logprob,
 * grad_entropy: [N] fp32, the latter NULL for 0 (entropy is then not read).
 * grad_logits: [N,V], I/O type, rows ld_grad apart; it may be the logits' own
 * buffer (with ld_grad = ld). */
LRS_API int lrs_logprobs_bwd(const void *logits, int64_t ld, const int64_t *target,
                             const float *lse, const float *entropy, const float *grad_logprob,
                             const float *grad_entropy, void *grad_logits, int64_t ld_grad,
                             int64_t N, int64_t V, int io_dtype, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LRS_BLOCK_H */
