/*
 * logra_policy.h - C ABI of the operators around the sketch in one policy
 * step, on AMD Instinct MI355X (gfx950): log probabilities of given tokens
 * with entropy and top alternatives, their gradient down to the logits, AdamW
 * over many tensors (the parameters that are not sketched), and the rank-r
 * updates of several policies applied to a layer's output without merging.
 *
 * Same library (liblogra.so), status codes and conventions as logra.h:
 * row-major matrices, caller-owned device buffers, no allocation, no state
 * between calls, work enqueued on `stream`, every argument that the host can
 * see checked before any HIP call, no synchronisation.  None of the entry
 * points records a memset, so all of them can be captured in a HIP graph
 * (host scalars are then fixed at their values of the capture: what that means for
 * an optimizer's step stands at logra_adamw_step).
 */
#ifndef LOGRA_POLICY_H
#define LOGRA_POLICY_H

#include "logra.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the entry points that take more than one. */
#define LOGRA_BF16 0
#define LOGRA_F32 1

/* Largest number of alternatives per row logra_token_logprob returns. */
#define LOGRA_MAX_TOP 64

/* Bytes of workspace logra_token_logprob needs (0 where it needs none: many
 * rows, or invalid sizes). */
size_t logra_token_logprob_ws_bytes(int64_t n_tok, int64_t vocab, int32_t n_top);

/*
 * logra_token_logprob - log probabilities of given tokens, with the entropy of
 * their distribution and its most probable tokens.
 *
 * For every row t, with a = z[t] / tau and p = softmax(a):
 *   lse[t]     = log sum_j e^a_j
 *   logp[t]    = a[target[t]] - lse[t]
 *   entropy[t] = -sum_j p_j log p_j        (0 log 0 = 0)
 *   top_idx[t, i], top_logp[t, i], i < n_top: the tokens with the largest
 *     logits in descending order, equal logits in ascending order of their
 *     index, and their log probabilities.
 * One pass over the logits; sums are held in fp32 about a running maximum.  Logits
 * may be of any finite size (masks of -1e30 or of the type's lowest value among
 * them): values that z / tau takes past fp32's range count as infinitely far, and
 * an lse or a log probability past it is infinite.
 *
 * Rows left out: a target outside [0, vocab) (e.g. -100 at a padded position)
 * marks a row whose logits are not read: logp, entropy and lse are 0,
 * top_idx -1 and top_logp -inf.
 * Masked tokens: a logit of -inf is a token of probability zero.  It is no
 * alternative: where fewer than n_top tokens have a logit above -inf the
 * remaining places hold -1 and -inf.  A target at such a token has logp -inf.
 * A row with no logit above -inf has lse -inf and logp and entropy NaN; a row
 * with a NaN or +inf logit has NaN in all of its values.  A NaN logit is no
 * alternative.
 *
 * z: device matrix [n_tok x ld] of `dtype` (LOGRA_BF16 or LOGRA_F32), ld >=
 *     vocab, ld % 8 == 0 (LOGRA_F32: ld % 4 == 0), 16-B aligned.
 * target: device int64[n_tok], 8-B aligned, or NULL: no row is left out, and
 *     logp must be NULL.
 * tau > 0, tau and 1.5 / tau finite; 0 <= n_top <= LOGRA_MAX_TOP.
 * logp, entropy, lse: device float[n_tok] or NULL, where not wanted.
 * top_idx: device int32[n_tok x n_top], top_logp: device float[n_tok x n_top];
 *     not inspected when n_top is 0.
 * ws: device scratch of logra_token_logprob_ws_bytes(n_tok, vocab, n_top)
 *     bytes, 256-B aligned (not inspected when that is 0).
 * Outputs, ws and inputs must not overlap.  0 <= n_tok < 2^31 (0: a no-op),
 * 1 <= vocab < 2^31.
 * Returns LOGRA_OK, LOGRA_EINVAL, LOGRA_EWORKSPACE or LOGRA_EHIP.
 */
int logra_token_logprob(const void* z, int dtype, int64_t n_tok, int64_t vocab, int64_t ld,
                        const int64_t* target, float tau, int32_t n_top, float* logp,
                        float* entropy, float* lse, int32_t* top_idx, float* top_logp, void* ws,
                        size_t ws_bytes, hipStream_t s);

/*
 * logra_token_logprob_backward - the gradient of a loss on logp, entropy and
 * lse down to the logits:
 *   dz_j = (d_logp ([j = target] - p_j) - d_entropy p_j (log p_j + entropy)
 *           + d_lse p_j) / tau,    log p_j = z_j / tau - lse
 * computed in fp32 and rounded once to dtype (bf16: to nearest even).  log p_j
 * carries the rounding of lse (2^-24 of it) and is held to at most 0: in rows so far
 * from zero that lse resolves whole units only, p_j is off by such a factor but stays
 * in [0, 1].
 * Rows left out (a target outside [0, vocab)) get zeros.  Masked tokens
 * (z = -inf, or so low that z / tau is) get zero, but for the d_logp of a masked
 * target.  Rows whose lse is not finite give NaN.  The factors d_logp / tau, d_lse /
 * tau and d_entropy (entropy + 128) / tau have to lie inside fp32's range: past it a
 * row holds infinities and NaN.
 *
 * z, dtype, n_tok, vocab, ld, target, tau: as in logra_token_logprob.
 * lse: device float[n_tok] of the forward call; entropy: likewise, needed only
 *     with d_entropy (NULL otherwise).
 * d_logp, d_entropy, d_lse: device float[n_tok] or NULL (zero), at least one
 *     given; d_logp needs target.
 * dz: device matrix [n_tok x ldz] of dtype, rules of z; elements past vocab
 *     are not written.  dz may be z itself with ldz == ld (the gradient then
 *     replaces the logits); no other overlap.
 * n_tok == 0 is a no-op.
 * Returns LOGRA_OK, LOGRA_EINVAL or LOGRA_EHIP.
 */
int logra_token_logprob_backward(const void* z, int dtype, int64_t n_tok, int64_t vocab,
                                 int64_t ld, const int64_t* target, float tau, const float* lse,
                                 const float* entropy, const float* d_logp,
                                 const float* d_entropy, const float* d_lse, void* dz,
                                 int64_t ldz, hipStream_t s);

/* Entries of an 8-bit state block, which share one exponent byte. */
#define LOGRA_STATE_BLOCK 32

/* One tensor of an AdamW step, n entries in each array. */
typedef struct logra_adamw_item {
  void* p;             /* weights, in/out: p_type */
  const void* g;       /* gradient: g_type */
  float* master;       /* fp32 weights behind a bf16 p, in/out, or NULL */
  void* m;             /* first moment, in/out: float[n], or uint8[n] codes */
  void* v;             /* second moment, in/out: float[n], or uint8[n] codes */
  uint8_t* m_exp;      /* 8-bit states: uint8[ceil(n / 32)] block exponents, in/out */
  uint8_t* v_exp;      /*   (fp32 states: NULL both) */
  int64_t n;
  float weight_decay;
  int32_t p_type;      /* LOGRA_BF16 or LOGRA_F32 */
  int32_t g_type;      /* LOGRA_BF16 or LOGRA_F32 */
} logra_adamw_item;

/* Bytes of a table of n tensors (0 for n < 0 or n > 2^24). */
size_t logra_adamw_table_bytes(int32_t n);

/*
 * logra_adamw_table - checks n tensors and lays them out for logra_adamw_step:
 * a host function, no HIP call.  A program makes the table once and again when
 * an array moves (the table holds addresses), and copies its bytes to device
 * memory.
 * items: host array of n entries, 0 <= n <= 2^24 (tensors with n == 0 entries are
 *     left out).  p, g, master, m, v aligned to their types; weight_decay
 *     finite.  No array that is written may overlap another (not checked).
 * table: host memory of logra_adamw_table_bytes(n) bytes, 8-B aligned, written.
 * Returns LOGRA_OK, LOGRA_EINVAL (also past 2^24 work-groups of one form, about
 * 6 10^10 entries) or LOGRA_EWORKSPACE (bytes too few).
 */
int logra_adamw_table(int32_t n, const logra_adamw_item* items, void* table, size_t bytes);

/*
 * logra_adamw_step - one AdamW step over the tensors of a table, one launch for
 * each form among them (weights, gradient and state types):
 *   g' = g grad_scale            (grad_scale: device float, NULL for 1)
 *   m <- beta1 m + (1 - beta1) g'
 *   v <- beta2 v + (1 - beta2) g'^2
 *   w <- w - lr ((m / b1) / (sqrt(v / b2) + eps) + weight_decay w)
 *   b1 = 1 - beta1^step, b2 = 1 - beta2^step
 * (Kingma & Ba, ICLR 2015, Algorithm 1, with the decay apart from the
 * gradient: Loshchilov & Hutter, ICLR 2019, Algorithm 2).  It is for the
 * parameters that are not sketched (norms, biases, embeddings);
 * logra_sketch_update holds the rules on a sketch.  Arithmetic is fp32 per
 * entry; 1 - beta and the bias corrections are formed in double and rounded
 * once.  w is master where given (p then gets w rounded to bf16), else p
 * itself; a bf16 p without a master is rounded to nearest even, so steps
 * smaller than half its spacing are lost.  The update uses the new m and v as
 * computed, before they are rounded to 8 bits.
 *
 * 8-bit states: blocks of 32 consecutive entries (the last one may be short)
 * share an exponent byte E, 16 <= E <= 254.  With bits(x) the fp32 pattern:
 *   m: sign in bit 7, c in bits 0..6, |m| = float((E - 15) << 23 | c << 20)
 *   v: c in bits 0..7, sqrt(v) = float((E - 15) << 23 | c << 19)
 *   (the two parts are added; c = 0 is zero), so an entry keeps 3 or 4
 *   mantissa bits over 16 binades below the block's largest; smaller m are
 *   zero, smaller nonzero sqrt(v) the least value (so that no division by a
 *   vanished v arises).  E = 255 marks a block with a NaN or an infinity (or
 *   past the largest finite value): all of its entries read as NaN.
 *   Rounding: bits(x) plus a dither below the bits kept, then truncated.  The
 *   dither of entry i of tensor j is the top 20 (m) or 19 (v) bits of
 *     h = (i + 32 B_j) 0x6A09E667 + step 0x9E3779B9 (+ 2^31 for v) mod 2^32,
 *   B_j the blocks of the tensors before j in the list.  Over steps it takes
 *   equally spaced values, so that states move by less than a rounding step on
 *   average as they should; rounded to nearest, a v with beta2 = 0.999 stays
 *   where it is (0.1 % of a step against a spacing of 6 %).
 *   Zeroed codes with any E below 255 are the zero state.
 *
 * In a captured graph lr, step and with it the bias corrections and the dither keep
 * the values of the capture at every replay.  Past the first steps, with the bias
 * corrections near 1, fp32 states do not need them to move; 8-bit states do: under
 * one and the same dither they are rounded with a bias, so this call stays outside
 * a graph there (or in as many graphs as there are steps).
 *
 * table: host memory as logra_adamw_table left it; table_dev: device copy of the
 *     same bytes, 8-B aligned (not inspected when there is nothing to do).
 * lr, eps finite as floats and >= 0 (with eps 0, also as a float, an entry whose v is
 *     zero becomes NaN); beta1, beta2 in [0, 1) as floats; step >= 1.
 * Returns LOGRA_OK, LOGRA_EINVAL or LOGRA_EHIP.
 */
int logra_adamw_step(const void* table, const void* table_dev, double lr, double beta1,
                     double beta2, double eps, int64_t step, const float* grad_scale,
                     hipStream_t s);

/* Which state logra_adamw_state_values reads. */
#define LOGRA_STATE_M 0
#define LOGRA_STATE_V 1

/*
 * logra_adamw_state_values - the values of an 8-bit state: m, or sqrt(v) for
 * LOGRA_STATE_V, as bf16 (which holds every value of the form exactly).
 * codes: device uint8[n]; exps: device uint8[ceil(n / 32)]; out: device
 * bf16[n], 2-B aligned; no overlap.  n == 0 is a no-op.
 * Returns LOGRA_OK, LOGRA_EINVAL or LOGRA_EHIP.
 */
int logra_adamw_state_values(int which, const uint8_t* codes, const uint8_t* exps, int64_t n,
                             uint16_t* out, hipStream_t s);

/* Bytes of workspace logra_adapter_apply needs.  Returns 0 for invalid sizes
 * (also past what one launch covers, about T d = 5 10^11) and for T == 0. */
size_t logra_adapter_ws_bytes(int64_t T, int64_t d, int64_t k, int32_t r);

/*
 * logra_adapter_apply - rank-r updates of n policies, unmerged, beside the
 * projection that they share:
 *   out[t] = RNE_bf16(Y[t] + c scale[a] (X[t] A_a^T) U_a^T),  a = adapter[t]
 * for every row t whose a lies in [0, n); other rows (-1: the base policy)
 * keep the bits of Y[t].  [LoGRA] Sketch / Sync: the update of a layer is
 * W - alpha eta U A with A rebuilt from a seed, and the payload of a policy is
 * (U, seed); with scale = -alpha eta, out is the layer's output under the
 * merged weights for a Y = X W^T of the shared ones, so that requests of
 * several policy versions run as one batch and a proposal's logits can be
 * formed with W left alone.  Rows of one policy need not be adjacent (tiles of
 * 32 rows with one policy are fastest).  P = X A^T is held in fp32 and enters
 * the second product as a bf16 pair of 16 significant bits, and so do fp32 U
 * (infinities, and values within 2^-9 of fp32's largest, come out as NaN).  A NaN
 * or an infinity in a row's X touches that row alone, one in a policy its rows.
 *
 * X: device bf16[T x ldx], k columns; Y, out: device bf16[T x ldy] / [T x
 *     ldo], d columns; ld rules of logra.h.  out may be Y itself with the same
 *     stride; columns past d are not written.  X, U, A must not overlap out.
 * adapter: device int32[T], 4-B aligned.
 * U: device [n x d x r] of u_type (LOGRA_F32 or LOGRA_BF16), contiguous,
 *     aligned to its type.
 * seeds: device uint64[n x 2] (seed, stream) of the sign basis, 8-B aligned;
 *     then c = 1 / sqrt(r) and A must be NULL.
 * A: else device bf16[n x r x lda] (row stride lda >= k; policies r lda apart;
 *     2-B aligned, fastest where rows lie on 16-byte boundaries): the bases
 *     themselves (e.g. Gaussian ones made once by logra_regen_A), c = 1, seeds
 *     NULL.
 * scale: device float[n], 4-B aligned.
 * ws: device scratch of logra_adapter_ws_bytes(T, d, k, r) bytes, 256-B
 *     aligned.
 * T == 0 is a no-op.  1 <= r <= LOGRA_MAX_RANK, 1 <= n < 2^31, d, k >= 1, all
 * of T, d, k < 2^31.  The same call gives the same bits.  A row that moves to
 * another tile of 32 rows, or into a batch of another size, may see its fp32 sums
 * over k in another order (tiles start at different columns, few tiles are cut
 * along k); moved inside its tile it keeps its bits.
 * Returns LOGRA_OK, LOGRA_EINVAL, LOGRA_EWORKSPACE or LOGRA_EHIP.
 */
int logra_adapter_apply(const uint16_t* X, int64_t ldx, const uint16_t* Y, int64_t ldy,
                        uint16_t* out, int64_t ldo, int64_t T, int64_t d, int64_t k, int32_t r,
                        int64_t n, const int32_t* adapter, const void* U, int u_type,
                        const uint64_t* seeds, const uint16_t* A, int64_t lda,
                        const float* scale, void* ws, size_t ws_bytes, hipStream_t s);

#ifdef __cplusplus
}
#endif

#endif /* LOGRA_POLICY_H */
