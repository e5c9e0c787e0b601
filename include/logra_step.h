/*
 * logra_step.h - C ABI of the operators that close a policy step, on AMD
 * Instinct MI355X (gfx950): drawing tokens from logits (the rollout), the layer
 * product with bias, activation and residual in its epilogue and its gradients
 * (what the sketch and the unmerged updates stand beside), and the global norm
 * of many gradients with clipping (what an optimizer's step is scaled by).
 *
 * Same library (liblogra.so), status codes and conventions as logra.h and
 * logra_policy.h: row-major matrices, rows on 16-byte boundaries, caller-owned
 * device buffers, no allocation, no state between calls, work enqueued on
 * `stream`, every argument that the host can see checked before any HIP call,
 * no synchronisation.  None of the entry points records a memset, so all of
 * them can be captured in a HIP graph (host scalars then keep the values of the
 * capture).  The same call gives the same bits.
 */
#ifndef LOGRA_STEP_H
#define LOGRA_STEP_H

#include "logra_policy.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ sampling */

/* Bytes of workspace logra_sample_tokens needs (0 where it needs none: many
 * rows, or invalid sizes). */
size_t logra_sample_tokens_ws_bytes(int64_t n_tok, int64_t vocab);

/*
 * logra_sample_tokens - one token per row of logits from a given random number,
 * with temperature, top-k, top-p and min-p.
 *
 * Row t, with a = z[t] / tau and p = softmax(a).  Its tokens with a logit above
 * -inf stand in descending order of their logits, equal ones in ascending order
 * of their index.  Kept are the first K of them, at least one:
 *   K1: the first top_k (top_k <= 0: all); M1 their mass (sum of p)
 *   Kp: the fewest with mass >= top_p M1 (top_p >= 1: no limit)
 *   Km: those with p_j >= min_p max p (min_p = 0: no limit)
 *   K = max(1, min(K1, Kp, Km)), M the mass of the first K.
 * token[t] is the first of this order whose cumulative mass exceeds u[t] M: for u
 * uniform in [0, 1) a draw from the kept tokens with probabilities p_j / M.
 * top_k = 1 is the most probable token.
 *   logp[t] = log p_token: what logra_token_logprob gives for that target
 *   logq[t] = log (p_token / M): the probability it was drawn with
 *   kept[t] = K
 * Masses are exact to about 2^-44 of each up to vocabularies of 2^18, to vocab 2^-62
 * past that (2^-31 at 2^31 tokens): fp64 exponentials, added as integers, so in no order, of
 * as many bits as let a sum of vocab of them fit.  A draw differs from one in exact
 * arithmetic only where u M lies that near to a border.
 *
 * A row with u[t] outside [0, 1) (an ended sequence: -1) is left out: token -1,
 * logp, logq and kept 0, its logits not read.  A row with a NaN or +inf logit,
 * with none above -inf, or with a setting outside its range has no token: -1, NaN,
 * NaN, 0.
 *
 * z, dtype, n_tok, vocab, ld: as in logra_token_logprob.
 * u: device float[n_tok].
 * tau, top_k, top_p, min_p: for all rows; tau > 0 finite, top_k >= 0, 0 < top_p
 *     <= 1, 0 <= min_p <= 1.  tau_rows, top_p_rows, min_p_rows: device
 *     float[n_tok], top_k_rows: device int32[n_tok], or NULL; where given, each
 *     row has its own and the scalar is not looked at.
 * token: device int64[n_tok]; logp, logq: device float[n_tok] or NULL; kept:
 *     device int32[n_tok] or NULL.
 * ws: device scratch of logra_sample_tokens_ws_bytes(n_tok, vocab) bytes, 256-B
 *     aligned (not inspected when that is 0).
 * Outputs, ws and inputs must not overlap.  n_tok == 0 is a no-op.
 * Returns LOGRA_OK, LOGRA_EINVAL, LOGRA_EWORKSPACE or LOGRA_EHIP.
 */
int logra_sample_tokens(const void* z, int dtype, int64_t n_tok, int64_t vocab, int64_t ld,
                        const float* u, float tau, int32_t top_k, float top_p, float min_p,
                        const float* tau_rows, const int32_t* top_k_rows,
                        const float* top_p_rows, const float* min_p_rows, int64_t* token,
                        float* logp, float* logq, int32_t* kept, void* ws, size_t ws_bytes,
                        hipStream_t s);

/* ------------------------------------------------------------------ gradient norm */

/* One tensor of n entries. */
typedef struct logra_grad_item {
  void* g;            /* gradient: g_type; written by logra_grad_clip where out is NULL */
  void* out;          /* what logra_grad_clip writes (out_type), or NULL */
  int64_t n;
  int32_t g_type;     /* LOGRA_BF16 or LOGRA_F32 */
  int32_t out_type;   /* LOGRA_BF16 or LOGRA_F32 (not looked at where out is NULL) */
} logra_grad_item;

/* Bytes of a table of n tensors (0 for n < 0 or n > 2^20). */
size_t logra_grad_table_bytes(int32_t n);

/*
 * logra_grad_table - checks n tensors and lays them out for logra_grad_norm and
 * logra_grad_clip: a host function, no HIP call.  A program makes the table once
 * and again when an array moves, and copies its bytes to device memory.
 * items: host array of n entries, 0 <= n <= 2^20.  Pointers aligned to their
 *     types.  out may be g itself with the same type; no other overlap of
 *     anything written (not checked).
 * table: host memory of logra_grad_table_bytes(n) bytes, 8-B aligned, written.
 * Returns LOGRA_OK, LOGRA_EINVAL or LOGRA_EWORKSPACE (bytes too few).
 */
int logra_grad_table(int32_t n, const logra_grad_item* items, void* table, size_t bytes);

/* Bytes of workspace logra_grad_norm needs for a table (0: not a table). */
size_t logra_grad_norm_ws_bytes(const void* table);

/* Which norm. */
#define LOGRA_NORM_2 0
#define LOGRA_NORM_INF 1

/*
 * logra_grad_norm - the norm of all entries of all tensors of a table, and the
 * factor that clips them:
 *   norm  = |s| (sum g^2)^(1/2), or |s| max |g| for LOGRA_NORM_INF
 *   scale = s min(1, max_norm / norm)
 *   norms[i]: the same norm of tensor i alone
 * s = grad_scale[0] (device float: a loss scale's inverse; NULL for 1).  scale is
 * what logra_adamw_step takes as its grad_scale.  Squares and sums are held in
 * fp64, which no fp32 gradient overflows.  A NaN entry makes norm and scale NaN; an
 * infinite one norm infinite and scale 0 (max_norm infinite: no clipping, scale = s).
 * Sketches S (d x r fp32) are tensors like others: E ||S||^2 = ||G||^2 for a
 * weight's gradient G under the bases of logra.h.
 *
 * table: host memory as logra_grad_table left it; table_dev: device copy of the
 *     same bytes, 8-B aligned (not inspected when no tensor has entries).
 * max_norm >= 0 (infinity: no clipping), not NaN.
 * norm, scale: device float[1] or NULL; norms: device float[n] or NULL, n the
 *     table's; at least one of the three given.
 * ws: device scratch of logra_grad_norm_ws_bytes(table) bytes, 256-B aligned.
 * Returns LOGRA_OK, LOGRA_EINVAL, LOGRA_EWORKSPACE or LOGRA_EHIP.
 */
int logra_grad_norm(const void* table, const void* table_dev, int kind, double max_norm,
                    const float* grad_scale, float* norm, float* scale, float* norms, void* ws,
                    size_t ws_bytes, hipStream_t s);

/*
 * logra_grad_clip - every tensor of a table times scale[0] (device float, as
 * logra_grad_norm left it): out = g scale in fp32, rounded to out's type (bf16: to
 * nearest even); in place where out is NULL, with nothing to do where scale is 1.
 * For gradients that no optimizer scales itself (logra_sketch_update, logra_merge).
 * scale lies in nothing that is written (not checked).
 * Returns LOGRA_OK, LOGRA_EINVAL or LOGRA_EHIP.
 */
int logra_grad_clip(const void* table, const void* table_dev, const float* scale, hipStream_t s);

/* ------------------------------------------------------------------ layer product */

/* Activations, as these formulas give them: +inf stays +inf, -inf is 0 under relu and
 * NaN (-inf times 0) under the others, NaN stays NaN. */
#define LOGRA_ACT_NONE 0
#define LOGRA_ACT_RELU 1        /* max(x, 0) */
#define LOGRA_ACT_SILU 2        /* x / (1 + e^-x) */
#define LOGRA_ACT_GELU 3        /* x Phi(x) */
#define LOGRA_ACT_GELU_TANH 4   /* x (1 + tanh(sqrt(2 / pi) (x + 0.044715 x^3))) / 2 */

/* Bytes of workspace that logra_linear, logra_linear_backward_input and
 * logra_linear_backward_weight need for a weight of d x k and T rows (enough for each
 * of the three; 0 where none is needed, or for invalid sizes), and that
 * logra_linear_backward_act needs with d_bias. */
size_t logra_linear_ws_bytes(int64_t T, int64_t d, int64_t k);
size_t logra_linear_backward_act_ws_bytes(int64_t T, int64_t d);

/*
 * logra_linear - a layer's product with its epilogue:
 *   pre = X W^T + bias,   out = act(pre) + residual
 * products and sums in fp32 on the matrix cores, act of the unrounded pre, one
 * rounding to out's type (bf16: to nearest even).
 *
 * X: device bf16[T x ldx], k columns; W: device bf16[d x ldw], k columns; ld rules
 *     of logra.h (multiples of 8, rows on 16-byte boundaries).
 * bias: device [d] of bias_type (LOGRA_BF16 or LOGRA_F32), or NULL.
 * residual: device bf16[T x ldr], d columns, or NULL; may be out itself (bf16, same
 *     stride).
 * out: device [T x ldo] of out_type, d columns (fp32: ldo a multiple of 4).
 * pre: device bf16[T x ldp], d columns: pre rounded, for the backward pass; or NULL.
 * Columns past d are not written.
 * ws: device scratch of logra_linear_ws_bytes(T, d, k) bytes, 256-B aligned (not
 *     inspected when that is 0).
 * No other overlap.  T == 0 is a no-op.  d, k >= 1; T, d, k < 2^31; results past what
 * one launch covers (about T d = 5 10^11) are refused.
 * Returns LOGRA_OK, LOGRA_EINVAL, LOGRA_EWORKSPACE or LOGRA_EHIP.
 */
int logra_linear(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw, int64_t T,
                 int64_t d, int64_t k, const void* bias, int bias_type, int act,
                 const uint16_t* residual, int64_t ldr, void* out, int out_type, int64_t ldo,
                 uint16_t* pre, int64_t ldp, void* ws, size_t ws_bytes, hipStream_t s);

/*
 * logra_linear_backward_act - the gradient of a loss from out back to pre, and to the
 * bias:
 *   dY = d_out act'(pre)  (rounded to bf16),   d_bias = sum over t of the unrounded dY
 * dY is what logra_sketch_accumulate, logra_linear_backward_input and
 * logra_linear_backward_weight take.  (A residual's gradient is d_out itself.)
 *
 * d_out: device [T x ldd] of d_out_type, d columns.  pre: device bf16[T x ldp] of
 *     logra_linear; NULL with LOGRA_ACT_NONE.  relu'(0) = 0.
 * dY: device bf16[T x ldy], or NULL (only d_bias is wanted); may be d_out itself (bf16,
 *     same stride) or pre itself (same stride).
 * d_bias: device float[d], written, or NULL; at least one of dY and d_bias given.
 * ws: with d_bias, device scratch of logra_linear_backward_act_ws_bytes(T, d) bytes,
 *     256-B aligned (not inspected when that is 0).
 * No other overlap.  T == 0: d_bias becomes zero.
 * Returns LOGRA_OK, LOGRA_EINVAL, LOGRA_EWORKSPACE or LOGRA_EHIP.
 */
int logra_linear_backward_act(const void* d_out, int d_out_type, int64_t ldd, const uint16_t* pre,
                              int64_t ldp, int act, int64_t T, int64_t d, uint16_t* dY,
                              int64_t ldy, float* d_bias, void* ws, size_t ws_bytes,
                              hipStream_t s);

/*
 * logra_linear_backward_input - dX = dY W + residual, rounded to bf16 once (residual:
 * device bf16[T x ldr], k columns, or NULL: a gradient that reaches X by another way,
 * e.g. past the layer; may be dX itself with the same stride).  Shapes as in
 * logra_linear; dX: device bf16[T x ldx], k columns.  ws of logra_linear_ws_bytes.
 * T == 0 is a no-op.
 */
int logra_linear_backward_input(const uint16_t* dY, int64_t ldy, const uint16_t* W, int64_t ldw,
                                int64_t T, int64_t d, int64_t k, const uint16_t* residual,
                                int64_t ldr, uint16_t* dX, int64_t ldx, void* ws,
                                size_t ws_bytes, hipStream_t s);

/* logra_linear_backward_weight: add to dW instead of writing it (fp32 only). */
#define LOGRA_LINEAR_ACCUMULATE 1

/*
 * logra_linear_backward_weight - dW = dY^T X, or dW += dY^T X: the full gradient, for
 * weights that are not sketched (a head, an embedding).  dW: device [d x ldw] of dw_type
 * (LOGRA_BF16 or LOGRA_F32), k columns.  flags: 0 or LOGRA_LINEAR_ACCUMULATE (dw_type
 * LOGRA_F32).  ws of logra_linear_ws_bytes.  T == 0: dW becomes zero, or stays.
 */
int logra_linear_backward_weight(const uint16_t* dY, int64_t ldy, const uint16_t* X, int64_t ldx,
                                 int64_t T, int64_t d, int64_t k, int flags, void* dW, int dw_type,
                                 int64_t ldw, void* ws, size_t ws_bytes, hipStream_t s);

#ifdef __cplusplus
}
#endif

#endif /* LOGRA_STEP_H */
