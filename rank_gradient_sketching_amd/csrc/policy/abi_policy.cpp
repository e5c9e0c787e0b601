// C ABI of the policy-step operators (declared in include/logra_policy.h).
//
// Every entry point validates all of its arguments on the host before the
// first HIP call and returns a status code; nothing throws across the ABI.
#include "logra_policy.h"

#include <math.h>
#include <string.h>

#include "abi_checks.hpp"
#include "internal.hpp"
#include "policy/internal_policy.hpp"

namespace {

using namespace logra::checks;
using logra::hip_status;

static_assert(LOGRA_MAX_TOP == logra::kMaxTop, "alternatives per row");
static_assert(LOGRA_STATE_BLOCK == logra::kStateBlock, "entries per 8-bit block");

// The table of an AdamW step: its head, the items, their first work-groups.
constexpr uint64_t kTableMagic = 0x57414D4152474F4Cull;
size_t table_bytes(int32_t n) {
  return (size_t)logra::round_up(
      (int64_t)sizeof(logra::AdamwTable) + (int64_t)n * ((int64_t)sizeof(logra::AdamwItem) + 4), 256);
}
static_assert(sizeof(logra::AdamwTable) % 8 == 0 && sizeof(logra::AdamwItem) % 8 == 0,
              "items on 8-byte boundaries");

}  // namespace

extern "C" {

size_t logra_token_logprob_ws_bytes(int64_t n_tok, int64_t vocab, int32_t n_top) {
  if (n_tok < 0 || n_tok >= kDimLimit || !dim_ok(vocab) || n_top < 0 || n_top > LOGRA_MAX_TOP)
    return 0;
  return logra::make_logprob_plan(n_tok, vocab, n_top).total;
}

int logra_token_logprob(const void* z, int dtype, int64_t n_tok, int64_t vocab, int64_t ld,
                        const int64_t* target, float tau, int32_t n_top, float* logp,
                        float* entropy, float* lse, int32_t* top_idx, float* top_logp, void* ws,
                        size_t ws_bytes, hipStream_t s) {
  if (!type_ok(dtype) || !dim_ok(vocab) || n_tok < 0 || n_tok >= kDimLimit) return LOGRA_EINVAL;
  if (n_top < 0 || n_top > LOGRA_MAX_TOP) return LOGRA_EINVAL;
  if (!tau_ok(tau)) return LOGRA_EINVAL;
  if (!ld_ok(ld, vocab, dtype)) return LOGRA_EINVAL;
  if (n_tok == 0) return LOGRA_OK;
  if (z == nullptr || !aligned(z, 16)) return LOGRA_EINVAL;
  if (target != nullptr && !aligned(target, 8)) return LOGRA_EINVAL;
  if (logp != nullptr && target == nullptr) return LOGRA_EINVAL;
  if (!aligned(logp, 4) || !aligned(entropy, 4) || !aligned(lse, 4)) return LOGRA_EINVAL;
  if (n_top > 0 && (top_idx == nullptr || top_logp == nullptr || !aligned(top_idx, 4) ||
                    !aligned(top_logp, 4)))
    return LOGRA_EINVAL;
  const logra::LogprobPlan p = logra::make_logprob_plan(n_tok, vocab, n_top);
  if (p.total > 0 && (ws == nullptr || ws_bytes < p.total || !aligned(ws, 256)))
    return LOGRA_EWORKSPACE;
  const Span all[8] = {span(logp, 1, n_tok, 0, 4),
                       span(entropy, 1, n_tok, 0, 4),
                       span(lse, 1, n_tok, 0, 4),
                       span(n_top ? top_idx : nullptr, n_tok, n_top, n_top, 4),
                       span(n_top ? top_logp : nullptr, n_tok, n_top, n_top, 4),
                       span(p.total ? ws : nullptr, 1, (int64_t)p.total, 0, 1),
                       span(z, n_tok, vocab, ld, bytes_of(dtype)),
                       span(target, 1, n_tok, 0, 8)};
  for (int i = 0; i < 6; ++i)
    for (int j = i + 1; j < 8; ++j)
      if (overlap(all[i], all[j])) return LOGRA_EINVAL;
  const logra::LogprobArgs a{z,    ld,      n_tok, (int)vocab, target,  tau, n_top,
                             logp, entropy, lse,   top_idx,    top_logp};
  return hip_status(
      logra::launch_token_logprob(a, dtype == LOGRA_F32, p, static_cast<char*>(ws), s));
}

int logra_token_logprob_backward(const void* z, int dtype, int64_t n_tok, int64_t vocab,
                                 int64_t ld, const int64_t* target, float tau, const float* lse,
                                 const float* entropy, const float* d_logp,
                                 const float* d_entropy, const float* d_lse, void* dz,
                                 int64_t ldz, hipStream_t s) {
  if (!type_ok(dtype) || !dim_ok(vocab) || n_tok < 0 || n_tok >= kDimLimit) return LOGRA_EINVAL;
  if (!tau_ok(tau)) return LOGRA_EINVAL;
  if (!ld_ok(ld, vocab, dtype) || !ld_ok(ldz, vocab, dtype)) return LOGRA_EINVAL;
  if (n_tok == 0) return LOGRA_OK;
  if (z == nullptr || dz == nullptr || lse == nullptr) return LOGRA_EINVAL;
  if (!aligned(z, 16) || !aligned(dz, 16) || !aligned(lse, 4)) return LOGRA_EINVAL;
  if (d_logp == nullptr && d_entropy == nullptr && d_lse == nullptr) return LOGRA_EINVAL;
  if (d_logp != nullptr && target == nullptr) return LOGRA_EINVAL;
  if (d_entropy != nullptr && entropy == nullptr) return LOGRA_EINVAL;
  if (!aligned(target, 8) || !aligned(entropy, 4) || !aligned(d_logp, 4) ||
      !aligned(d_entropy, 4) || !aligned(d_lse, 4))
    return LOGRA_EINVAL;
  const int64_t e = bytes_of(dtype);
  const Span out = span(dz, n_tok, vocab, ldz, e);
  const Span in = span(z, n_tok, vocab, ld, e);
  if (out.hi == kNoEnd || (!(dz == z && ldz == ld) && overlap(out, in))) return LOGRA_EINVAL;
  const void* rows[5] = {lse, d_entropy ? entropy : nullptr, d_logp, d_entropy, d_lse};
  for (const void* q : rows)
    if (overlap(out, span(q, 1, n_tok, 0, 4))) return LOGRA_EINVAL;
  if (overlap(out, span(target, 1, n_tok, 0, 8))) return LOGRA_EINVAL;
  const logra::LogprobGradArgs a{z,       ld,     n_tok,     (int)vocab, target, tau, lse,
                                 entropy, d_logp, d_entropy, d_lse,      dz,     ldz};
  return hip_status(logra::launch_token_logprob_backward(a, dtype == LOGRA_F32, s));
}

size_t logra_adamw_table_bytes(int32_t n) {
  if (n < 0 || n > (1 << 24)) return 0;
  return table_bytes(n);
}

int logra_adamw_table(int32_t n, const logra_adamw_item* items, void* table, size_t bytes) {
  if (n < 0 || n > (1 << 24) || (n > 0 && items == nullptr)) return LOGRA_EINVAL;
  if (table == nullptr || !aligned(table, 8)) return LOGRA_EINVAL;
  if (bytes < table_bytes(n)) return LOGRA_EWORKSPACE;
  for (int i = 0; i < n; ++i) {
    const logra_adamw_item& q = items[i];
    if (!type_ok(q.p_type) || !type_ok(q.g_type) || !isfinite(q.weight_decay)) return LOGRA_EINVAL;
    if (q.n < 0 || q.n >= kLdLimit) return LOGRA_EINVAL;
    const bool state8 = q.m_exp != nullptr;
    if (state8 != (q.v_exp != nullptr)) return LOGRA_EINVAL;
    if (q.master != nullptr && q.p_type == LOGRA_F32) return LOGRA_EINVAL;
    if (q.n == 0) continue;
    if (q.p == nullptr || q.g == nullptr || q.m == nullptr || q.v == nullptr) return LOGRA_EINVAL;
    if (!aligned(q.p, bytes_of(q.p_type)) || !aligned(q.g, bytes_of(q.g_type)) ||
        !aligned(q.master, 4) || !aligned(q.m, state8 ? 1 : 4) || !aligned(q.v, state8 ? 1 : 4))
      return LOGRA_EINVAL;
  }
  char* const base = static_cast<char*>(table);
  memset(base, 0, table_bytes(n));
  logra::AdamwTable* const t = reinterpret_cast<logra::AdamwTable*>(base);
  t->magic = kTableMagic;
  t->bytes = table_bytes(n);
  auto form_of = [](const logra_adamw_item& q) {
    const int weights = q.p_type == LOGRA_F32 ? 0 : q.master == nullptr ? 1 : 2;
    return weights * 4 + (q.g_type == LOGRA_F32 ? 2 : 0) + (q.m_exp != nullptr ? 1 : 0);
  };
  for (int i = 0; i < n; ++i)
    if (items[i].n > 0) ++t->form[form_of(items[i])].n;
  // the items of all forms, then their first work-groups
  uint32_t at = sizeof(logra::AdamwTable);
  for (logra::AdamwForm& f : t->form) {
    f.off_items = at;
    at += (uint32_t)f.n * (uint32_t)sizeof(logra::AdamwItem);
  }
  for (logra::AdamwForm& f : t->form) {
    f.off_first = at;
    at += (uint32_t)f.n * 4;
  }
  int32_t done[logra::kAdamwForms] = {};
  uint32_t dither0 = 0;
  for (int i = 0; i < n; ++i) {
    const logra_adamw_item& x = items[i];
    if (x.n == 0) continue;
    const int k = form_of(x);
    reinterpret_cast<logra::AdamwItem*>(base + t->form[k].off_items)[done[k]++] =
        logra::AdamwItem{x.p, x.g, x.master, x.m, x.v, x.m_exp, x.v_exp, x.n, x.weight_decay,
                         dither0, 0, 0};
    dither0 += (uint32_t)logra::round_up(x.n, logra::kStateBlock);
  }
  for (int k = 0; k < logra::kAdamwForms; ++k) {
    logra::AdamwForm& f = t->form[k];
    if (!logra::adamw_lay_out(&f, reinterpret_cast<logra::AdamwItem*>(base + f.off_items),
                              reinterpret_cast<int32_t*>(base + f.off_first), (k & 2) != 0,
                              (k & 1) != 0, static_cast<logra::AdamwWeights>(k / 4))) {
      t->magic = 0;
      return LOGRA_EINVAL;
    }
  }
  return LOGRA_OK;
}

int logra_adamw_step(const void* table, const void* table_dev, double lr, double beta1,
                     double beta2, double eps, int64_t step, const float* grad_scale,
                     hipStream_t s) {
  if (table == nullptr || !aligned(table, 8)) return LOGRA_EINVAL;
  const logra::AdamwTable& t = *static_cast<const logra::AdamwTable*>(table);
  if (t.magic != kTableMagic) return LOGRA_EINVAL;
  if (!isfinite((float)lr) || lr < 0.0 || !isfinite((float)eps) || eps < 0.0 || step < 1)
    return LOGRA_EINVAL;
  for (const double b : {beta1, beta2})
    if (!isfinite(b) || b < 0.0 || !((float)b < 1.0f)) return LOGRA_EINVAL;
  if (!aligned(grad_scale, 4)) return LOGRA_EINVAL;
  bool any = false;
  for (const logra::AdamwForm& f : t.form) any = any || f.n > 0;
  if (!any) return LOGRA_OK;
  if (table_dev == nullptr || !aligned(table_dev, 8)) return LOGRA_EINVAL;
  logra::AdamwScalars h{};
  h.lr = (float)lr;
  h.b1 = (float)beta1;
  h.b2 = (float)beta2;
  h.c1 = (float)(1.0 - beta1);
  h.c2 = (float)(1.0 - beta2);
  h.eps = (float)eps;
  h.inv_bc1 = (float)(1.0 / (1.0 - pow(beta1, (double)step)));
  h.inv_sqrt_bc2 = (float)(1.0 / sqrt(1.0 - pow(beta2, (double)step)));
  h.dither_step = (uint32_t)step * logra::kDitherStep;
  h.grad_scale = grad_scale;
  const char* const dev = static_cast<const char*>(table_dev);
  for (int k = 0; k < logra::kAdamwForms; ++k) {
    const logra::AdamwForm& f = t.form[k];
    if (f.n == 0) continue;
    const int st = hip_status(logra::launch_adamw(
        static_cast<logra::AdamwWeights>(k / 4), (k & 2) != 0, (k & 1) != 0, f,
        reinterpret_cast<const logra::AdamwItem*>(dev + f.off_items),
        reinterpret_cast<const int32_t*>(dev + f.off_first), h, s));
    if (st != LOGRA_OK) return st;
  }
  return LOGRA_OK;
}

int logra_adamw_state_values(int which, const uint8_t* codes, const uint8_t* exps, int64_t n,
                             uint16_t* out, hipStream_t s) {
  if (which != LOGRA_STATE_M && which != LOGRA_STATE_V) return LOGRA_EINVAL;
  if (n < 0 || n >= kLdLimit) return LOGRA_EINVAL;
  if (n == 0) return LOGRA_OK;
  if (codes == nullptr || exps == nullptr || out == nullptr || !aligned(out, 2))
    return LOGRA_EINVAL;
  const Span o = span(out, 1, n, 0, 2);
  if (overlap(o, span(codes, 1, n, 0, 1)) ||
      overlap(o, span(exps, 1, (n + LOGRA_STATE_BLOCK - 1) / LOGRA_STATE_BLOCK, 0, 1)))
    return LOGRA_EINVAL;
  return hip_status(
      logra::launch_adamw_state_values(which == LOGRA_STATE_V, codes, exps, n, out, s));
}

size_t logra_adapter_ws_bytes(int64_t T, int64_t d, int64_t k, int32_t r) {
  logra::AdapterPlan p{};
  return logra::make_adapter_plan(T, d, k, r, &p) ? p.total : 0;
}

int logra_adapter_apply(const uint16_t* X, int64_t ldx, const uint16_t* Y, int64_t ldy,
                        uint16_t* out, int64_t ldo, int64_t T, int64_t d, int64_t k, int32_t r,
                        int64_t n, const int32_t* adapter, const void* U, int u_type,
                        const uint64_t* seeds, const uint16_t* A, int64_t lda,
                        const float* scale, void* ws, size_t ws_bytes, hipStream_t s) {
  if (T < 0 || T >= kDimLimit || !dim_ok(d) || !dim_ok(k) || !dim_ok(n)) return LOGRA_EINVAL;
  if (r < 1 || r > LOGRA_MAX_RANK || !type_ok(u_type)) return LOGRA_EINVAL;
  if (!ld_ok(ldx, k, LOGRA_BF16) || !ld_ok(ldy, d, LOGRA_BF16) || !ld_ok(ldo, d, LOGRA_BF16))
    return LOGRA_EINVAL;
  if ((seeds == nullptr) == (A == nullptr)) return LOGRA_EINVAL;
  if (A != nullptr && (!aligned(A, 2) || lda < k || lda >= kLdLimit)) return LOGRA_EINVAL;
  if (seeds != nullptr && !aligned(seeds, 8)) return LOGRA_EINVAL;
  if (T == 0) return LOGRA_OK;
  if (X == nullptr || Y == nullptr || out == nullptr || adapter == nullptr || U == nullptr ||
      scale == nullptr)
    return LOGRA_EINVAL;
  if (!aligned(X, 16) || !aligned(Y, 16) || !aligned(out, 16) || !aligned(adapter, 4) ||
      !aligned(U, (uintptr_t)bytes_of(u_type)) || !aligned(scale, 4))
    return LOGRA_EINVAL;
  logra::AdapterPlan p{};
  if (!logra::make_adapter_plan(T, d, k, r, &p)) return LOGRA_EINVAL;
  if (ws == nullptr || ws_bytes < p.total || !aligned(ws, 256)) return LOGRA_EWORKSPACE;
  const Span o = span(out, T, d, ldo, 2), w = span(ws, 1, (int64_t)p.total, 0, 1);
  const Span y = span(Y, T, d, ldy, 2);
  if (!(out == Y && ldo == ldy) && overlap(o, y)) return LOGRA_EINVAL;
  const Span in[7] = {span(X, T, k, ldx, 2),
                      span(U, n * d, r, r, bytes_of(u_type)),
                      span(A, n * r, k, lda, 2),
                      span(adapter, 1, T, 0, 4),
                      span(scale, 1, n, 0, 4),
                      span(seeds, 1, 2 * n, 0, 8),
                      w};
  for (const Span& x : in)
    if (overlap(o, x)) return LOGRA_EINVAL;
  for (int i = 0; i < 6; ++i)
    if (overlap(w, in[i])) return LOGRA_EINVAL;
  if (overlap(w, y)) return LOGRA_EINVAL;
  const logra::AdapterArgs a{X,      ldx, Y, ldy,   out, ldo, T, (int)d, (int)k, (int)r, n,
                             adapter, U,  seeds, A, lda, scale};
  return hip_status(
      logra::launch_adapter(a, u_type == LOGRA_F32, p, static_cast<char*>(ws), s));
}

}  // extern "C"
