// C ABI of the operators that close a policy step (declared in
// include/logra_step.h).
//
// Every entry point validates all of its arguments on the host before the
// first HIP call and returns a status code; nothing throws across the ABI.
#include "logra_step.h"

#include <math.h>
#include <string.h>

#include "abi_checks.hpp"
#include "internal.hpp"
#include "step/internal_step.hpp"

namespace {

using namespace logra::checks;
using logra::hip_status;

static_assert(LOGRA_ACT_NONE == logra::kActNone && LOGRA_ACT_RELU == logra::kActRelu &&
                  LOGRA_ACT_SILU == logra::kActSilu && LOGRA_ACT_GELU == logra::kActGelu &&
                  LOGRA_ACT_GELU_TANH == logra::kActGeluTanh,
              "activations");

constexpr int32_t kMaxGrads = 1 << 20;
constexpr uint64_t kGradMagic = 0x4C4C415247524F4Cull;
size_t grad_bytes(int32_t n) {
  return (size_t)logra::round_up((int64_t)sizeof(logra::GradTable) +
                                     (int64_t)n * (int64_t)sizeof(logra::GradItem) +
                                     ((int64_t)n + 1) * 4,
                                 256);
}
static_assert(sizeof(logra::GradTable) % 8 == 0 && sizeof(logra::GradItem) % 8 == 0,
              "items on 8-byte boundaries");

const logra::GradTable* grad_head(const void* table) {
  if (table == nullptr || !aligned(table, 8)) return nullptr;
  const logra::GradTable* const t = static_cast<const logra::GradTable*>(table);
  return t->magic == kGradMagic ? t : nullptr;
}
logra::GradNormArgs grad_args(const logra::GradTable& t, const void* table_dev) {
  logra::GradNormArgs a{};
  const char* const dev = static_cast<const char*>(table_dev) + sizeof(logra::GradTable);
  a.items = reinterpret_cast<const logra::GradItem*>(dev);
  a.first = reinterpret_cast<const int32_t*>(dev + (size_t)t.n * sizeof(logra::GradItem));
  a.n = t.n;
  a.groups = t.groups;
  a.loops = t.loops;
  a.large = t.large != 0;
  return a;
}

// A matrix argument: its rows and columns, stride and type.
bool matrix_ok(const void* p, int64_t ld, int64_t cols, int type) {
  return p != nullptr && aligned(p, 16) && ld_ok(ld, cols, type);
}
bool ws_ok(size_t need, const void* ws, size_t bytes) {
  return need == 0 || (ws != nullptr && bytes >= need && aligned(ws, 256));
}
// A written span against what else the call touches.
bool any_overlap(const Span& out, const Span* in, int n) {
  if (out.hi == kNoEnd) return true;
  for (int i = 0; i < n; ++i)
    if (overlap(out, in[i])) return true;
  return false;
}
bool sizes_ok(int64_t T, int64_t d, int64_t k) {
  return T >= 0 && T < kDimLimit && dim_ok(d) && dim_ok(k);
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------ sampling
size_t logra_sample_tokens_ws_bytes(int64_t n_tok, int64_t vocab) {
  if (n_tok < 0 || n_tok >= kDimLimit || !dim_ok(vocab)) return 0;
  return logra::sample_ws_bytes(n_tok, vocab);
}

int logra_sample_tokens(const void* z, int dtype, int64_t n_tok, int64_t vocab, int64_t ld,
                        const float* u, float tau, int32_t top_k, float top_p, float min_p,
                        const float* tau_rows, const int32_t* top_k_rows,
                        const float* top_p_rows, const float* min_p_rows, int64_t* token,
                        float* logp, float* logq, int32_t* kept, void* ws, size_t ws_bytes,
                        hipStream_t s) {
  if (!type_ok(dtype) || !dim_ok(vocab) || n_tok < 0 || n_tok >= kDimLimit) return LOGRA_EINVAL;
  if (!ld_ok(ld, vocab, dtype)) return LOGRA_EINVAL;
  if (tau_rows == nullptr && !(tau > 0.0f && isfinite(tau))) return LOGRA_EINVAL;
  if (top_k_rows == nullptr && top_k < 0) return LOGRA_EINVAL;
  if (top_p_rows == nullptr && !(top_p > 0.0f && top_p <= 1.0f)) return LOGRA_EINVAL;
  if (min_p_rows == nullptr && !(min_p >= 0.0f && min_p <= 1.0f)) return LOGRA_EINVAL;
  if (n_tok == 0) return LOGRA_OK;
  if (z == nullptr || !aligned(z, 16) || u == nullptr || token == nullptr) return LOGRA_EINVAL;
  if (!aligned(token, 8)) return LOGRA_EINVAL;
  const void* const words[8] = {u,          tau_rows, top_k_rows, top_p_rows,
                                min_p_rows, logp,     logq,       kept};
  for (const void* p : words)
    if (!aligned(p, 4)) return LOGRA_EINVAL;
  const size_t need = logra::sample_ws_bytes(n_tok, vocab);
  if (!ws_ok(need, ws, ws_bytes)) return LOGRA_EWORKSPACE;
  Span all[11] = {span(token, 1, n_tok, 0, 8), span(logp, 1, n_tok, 0, 4),
                  span(logq, 1, n_tok, 0, 4),  span(kept, 1, n_tok, 0, 4),
                  span(need ? ws : nullptr, 1, (int64_t)need, 0, 1),
                  span(z, n_tok, vocab, ld, bytes_of(dtype))};
  for (int i = 0; i < 5; ++i) all[6 + i] = span(words[i], 1, n_tok, 0, 4);
  for (int i = 0; i < 5; ++i)
    if (any_overlap(all[i], all + i + 1, 10 - i)) return LOGRA_EINVAL;
  const logra::SampleArgs a{z,     ld,    n_tok,    (int)vocab, u,          tau,
                            top_k, top_p, min_p,    tau_rows,   top_k_rows, top_p_rows,
                            min_p_rows, token, logp, logq,      kept};
  return hip_status(logra::launch_sample(a, dtype == LOGRA_F32, static_cast<char*>(ws), s));
}

// ------------------------------------------------------------------ gradient norm
size_t logra_grad_table_bytes(int32_t n) { return n < 0 || n > kMaxGrads ? 0 : grad_bytes(n); }

int logra_grad_table(int32_t n, const logra_grad_item* items, void* table, size_t bytes) {
  if (n < 0 || n > kMaxGrads || (n > 0 && items == nullptr)) return LOGRA_EINVAL;
  if (table == nullptr || !aligned(table, 8)) return LOGRA_EINVAL;
  if (bytes < grad_bytes(n)) return LOGRA_EWORKSPACE;
  for (int i = 0; i < n; ++i) {
    const logra_grad_item& q = items[i];
    if (!type_ok(q.g_type) || q.n < 0 || q.n >= kLdLimit) return LOGRA_EINVAL;
    if (q.out != nullptr && !type_ok(q.out_type)) return LOGRA_EINVAL;
    if (q.n == 0) continue;
    if (q.g == nullptr || !aligned(q.g, bytes_of(q.g_type))) return LOGRA_EINVAL;
    if (q.out != nullptr && (!aligned(q.out, bytes_of(q.out_type)) ||
                             (q.out == q.g && q.out_type != q.g_type)))
      return LOGRA_EINVAL;
  }
  char* const base = static_cast<char*>(table);
  memset(base, 0, grad_bytes(n));
  logra::GradTable* const t = reinterpret_cast<logra::GradTable*>(base);
  logra::GradItem* const to = reinterpret_cast<logra::GradItem*>(base + sizeof(logra::GradTable));
  for (int i = 0; i < n; ++i) {
    const logra_grad_item& q = items[i];
    const bool in_place = q.out == nullptr;
    to[i] = logra::GradItem{q.g, in_place ? q.g : q.out, q.n, q.g_type == LOGRA_F32,
                            (in_place ? q.g_type : q.out_type) == LOGRA_F32, 0, 0};
  }
  t->n = n;
  t->bytes = grad_bytes(n);
  if (!logra::grad_lay_out(t, to, reinterpret_cast<int32_t*>(to + n))) return LOGRA_EINVAL;
  t->magic = kGradMagic;
  return LOGRA_OK;
}

size_t logra_grad_norm_ws_bytes(const void* table) {
  const logra::GradTable* const t = grad_head(table);
  return t == nullptr ? 0 : (size_t)logra::round_up((t->groups > 0 ? t->groups : 1) * 8, 256);
}

int logra_grad_norm(const void* table, const void* table_dev, int kind, double max_norm,
                    const float* grad_scale, float* norm, float* scale, float* norms, void* ws,
                    size_t ws_bytes, hipStream_t s) {
  const logra::GradTable* const t = grad_head(table);
  if (t == nullptr || (kind != LOGRA_NORM_2 && kind != LOGRA_NORM_INF)) return LOGRA_EINVAL;
  if (!(max_norm >= 0.0)) return LOGRA_EINVAL;
  if (t->n == 0) norms = nullptr;
  if (norm == nullptr && scale == nullptr && norms == nullptr)
    return t->n == 0 ? LOGRA_OK : LOGRA_EINVAL;
  if (!aligned(grad_scale, 4) || !aligned(norm, 4) || !aligned(scale, 4) || !aligned(norms, 4))
    return LOGRA_EINVAL;
  if (t->groups > 0 && (table_dev == nullptr || !aligned(table_dev, 8))) return LOGRA_EINVAL;
  const size_t need = logra_grad_norm_ws_bytes(table);
  if (!ws_ok(need, ws, ws_bytes)) return LOGRA_EWORKSPACE;
  const Span all[6] = {span(norm, 1, 1, 0, 4),
                       span(scale, 1, 1, 0, 4),
                       span(norms, 1, t->n, 0, 4),
                       span(ws, 1, (int64_t)need, 0, 1),
                       span(grad_scale, 1, 1, 0, 4),
                       span(t->groups > 0 ? table_dev : nullptr, 1, (int64_t)t->bytes, 0, 1)};
  for (int i = 0; i < 4; ++i)
    if (any_overlap(all[i], all + i + 1, 5 - i)) return LOGRA_EINVAL;
  logra::GradNormArgs a = grad_args(*t, table_dev);
  a.inf_norm = kind == LOGRA_NORM_INF;
  a.max_norm = max_norm;
  a.grad_scale = grad_scale;
  a.norm = norm;
  a.scale = scale;
  a.norms = norms;
  return hip_status(logra::launch_grad_norm(a, static_cast<double*>(ws), s));
}

int logra_grad_clip(const void* table, const void* table_dev, const float* scale, hipStream_t s) {
  const logra::GradTable* const t = grad_head(table);
  if (t == nullptr || scale == nullptr || !aligned(scale, 4)) return LOGRA_EINVAL;
  if (t->groups == 0) return LOGRA_OK;
  if (table_dev == nullptr || !aligned(table_dev, 8)) return LOGRA_EINVAL;
  return hip_status(logra::launch_grad_clip(grad_args(*t, table_dev), scale, s));
}

// ------------------------------------------------------------------ layer product
size_t logra_linear_ws_bytes(int64_t T, int64_t d, int64_t k) {
  if (!sizes_ok(T, d, k) || T == 0) return 0;
  const size_t a = logra::gemm_ws_bytes(logra::GemmForm::kForward, T, d, k);
  const size_t b = logra::gemm_ws_bytes(logra::GemmForm::kInput, T, k, d);
  const size_t c = logra::gemm_ws_bytes(logra::GemmForm::kWeight, d, k, T);
  return a > b ? (a > c ? a : c) : (b > c ? b : c);
}

size_t logra_linear_backward_act_ws_bytes(int64_t T, int64_t d) {
  if (T < 0 || T >= kDimLimit || !dim_ok(d)) return 0;
  return logra::act_grad_ws_bytes(T, d);
}

int logra_linear(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw, int64_t T,
                 int64_t d, int64_t k, const void* bias, int bias_type, int act,
                 const uint16_t* residual, int64_t ldr, void* out, int out_type, int64_t ldo,
                 uint16_t* pre, int64_t ldp, void* ws, size_t ws_bytes, hipStream_t s) {
  if (!sizes_ok(T, d, k) || act < 0 || act >= logra::kActs || !type_ok(out_type))
    return LOGRA_EINVAL;
  if (bias != nullptr && (!type_ok(bias_type) || !aligned(bias, (uintptr_t)bytes_of(bias_type))))
    return LOGRA_EINVAL;
  if (!ld_ok(ldx, k, LOGRA_BF16) || !ld_ok(ldw, k, LOGRA_BF16) || !ld_ok(ldo, d, out_type))
    return LOGRA_EINVAL;
  if (residual != nullptr && !matrix_ok(residual, ldr, d, LOGRA_BF16)) return LOGRA_EINVAL;
  if (pre != nullptr && !matrix_ok(pre, ldp, d, LOGRA_BF16)) return LOGRA_EINVAL;
  if (T == 0) return LOGRA_OK;
  if (!matrix_ok(X, ldx, k, LOGRA_BF16) || !matrix_ok(W, ldw, k, LOGRA_BF16) ||
      !matrix_ok(out, ldo, d, out_type))
    return LOGRA_EINVAL;
  if (!logra::gemm_fits(logra::GemmForm::kForward, T, d, k)) return LOGRA_EINVAL;
  const size_t need = logra::gemm_ws_bytes(logra::GemmForm::kForward, T, d, k);
  if (!ws_ok(need, ws, ws_bytes)) return LOGRA_EWORKSPACE;
  const Span o = span(out, T, d, ldo, bytes_of(out_type)), r = span(residual, T, d, ldr, 2);
  const Span p = span(pre, T, d, ldp, 2), w = span(need ? ws : nullptr, 1, (int64_t)need, 0, 1);
  const Span in[4] = {span(X, T, k, ldx, 2), span(W, d, k, ldw, 2),
                      span(bias, 1, d, 0, bytes_of(bias_type)), r};
  const bool same = residual == out && out_type == LOGRA_BF16 && ldr == ldo;
  if (any_overlap(o, in, same ? 3 : 4) || any_overlap(p, in, 4) || any_overlap(w, in, 4))
    return LOGRA_EINVAL;
  if (overlap(o, p) || overlap(o, w) || overlap(p, w)) return LOGRA_EINVAL;
  logra::GemmArgs g{};
  g.A = X;
  g.lda = ldx;
  g.B = W;
  g.ldb = ldw;
  g.M = (int)T;
  g.N = (int)d;
  g.K = (int)k;
  g.bias = bias;
  g.bias_f32 = bias_type == LOGRA_F32;
  g.act = act;
  g.add = residual;
  g.ldadd = ldr;
  g.C = out;
  g.ldc = ldo;
  g.c_f32 = out_type == LOGRA_F32;
  g.pre = pre;
  g.ldpre = ldp;
  return hip_status(
      logra::launch_gemm(logra::GemmForm::kForward, g, static_cast<char*>(ws), s));
}

int logra_linear_backward_act(const void* d_out, int d_out_type, int64_t ldd, const uint16_t* pre,
                              int64_t ldp, int act, int64_t T, int64_t d, uint16_t* dY,
                              int64_t ldy, float* d_bias, void* ws, size_t ws_bytes,
                              hipStream_t s) {
  if (T < 0 || T >= kDimLimit || !dim_ok(d) || act < 0 || act >= logra::kActs ||
      !type_ok(d_out_type))
    return LOGRA_EINVAL;
  if ((dY == nullptr && d_bias == nullptr) || (act == LOGRA_ACT_NONE && pre != nullptr))
    return LOGRA_EINVAL;
  if (!ld_ok(ldd, d, d_out_type) || !aligned(d_bias, 4)) return LOGRA_EINVAL;
  if (dY != nullptr && !matrix_ok(dY, ldy, d, LOGRA_BF16)) return LOGRA_EINVAL;
  if (act != LOGRA_ACT_NONE && !ld_ok(ldp, d, LOGRA_BF16)) return LOGRA_EINVAL;
  if (T == 0 && d_bias == nullptr) return LOGRA_OK;
  if (T > 0 && (d_out == nullptr || !aligned(d_out, 16))) return LOGRA_EINVAL;
  if (T > 0 && act != LOGRA_ACT_NONE && (pre == nullptr || !aligned(pre, 16))) return LOGRA_EINVAL;
  const size_t need = d_bias != nullptr ? logra::act_grad_ws_bytes(T, d) : 0;
  if (!ws_ok(need, ws, ws_bytes)) return LOGRA_EWORKSPACE;
  const Span y = span(dY, T, d, ldy, 2), b = span(d_bias, 1, d, 0, 4);
  const Span w = span(need ? ws : nullptr, 1, (int64_t)need, 0, 1);
  const Span g = span(T > 0 ? d_out : nullptr, T, d, ldd, bytes_of(d_out_type));
  const Span p = span(T > 0 ? pre : nullptr, T, d, ldp, 2);
  if (y.hi == kNoEnd || g.hi == kNoEnd || p.hi == kNoEnd) return LOGRA_EINVAL;
  if (overlap(y, g) && !(dY == d_out && d_out_type == LOGRA_BF16 && ldy == ldd))
    return LOGRA_EINVAL;
  if (overlap(y, p) && !(dY == pre && ldy == ldp)) return LOGRA_EINVAL;
  const Span rest[3] = {y, g, p};
  if (any_overlap(b, rest, 3) || any_overlap(w, rest, 3) || overlap(b, w)) return LOGRA_EINVAL;
  const logra::ActGradArgs a{d_out, d_out_type == LOGRA_F32, ldd, pre, ldp, act, T, (int)d, dY, ldy,
                             d_bias};
  return hip_status(logra::launch_act_grad(a, static_cast<char*>(ws), s));
}

int logra_linear_backward_input(const uint16_t* dY, int64_t ldy, const uint16_t* W, int64_t ldw,
                                int64_t T, int64_t d, int64_t k, const uint16_t* residual,
                                int64_t ldr, uint16_t* dX, int64_t ldx, void* ws,
                                size_t ws_bytes, hipStream_t s) {
  if (!sizes_ok(T, d, k)) return LOGRA_EINVAL;
  if (!ld_ok(ldy, d, LOGRA_BF16) || !ld_ok(ldw, k, LOGRA_BF16) || !ld_ok(ldx, k, LOGRA_BF16))
    return LOGRA_EINVAL;
  if (residual != nullptr && !matrix_ok(residual, ldr, k, LOGRA_BF16)) return LOGRA_EINVAL;
  if (T == 0) return LOGRA_OK;
  if (!matrix_ok(dY, ldy, d, LOGRA_BF16) || !matrix_ok(W, ldw, k, LOGRA_BF16) ||
      !matrix_ok(dX, ldx, k, LOGRA_BF16))
    return LOGRA_EINVAL;
  if (!logra::gemm_fits(logra::GemmForm::kInput, T, k, d)) return LOGRA_EINVAL;
  const size_t need = logra::gemm_ws_bytes(logra::GemmForm::kInput, T, k, d);
  if (!ws_ok(need, ws, ws_bytes)) return LOGRA_EWORKSPACE;
  const Span o = span(dX, T, k, ldx, 2), w = span(need ? ws : nullptr, 1, (int64_t)need, 0, 1);
  const Span in[3] = {span(dY, T, d, ldy, 2), span(W, d, k, ldw, 2),
                      span(residual, T, k, ldr, 2)};
  const bool same = residual == dX && ldr == ldx;
  if (any_overlap(o, in, same ? 2 : 3) || any_overlap(w, in, 3) || overlap(o, w))
    return LOGRA_EINVAL;
  logra::GemmArgs g{};
  g.A = dY;
  g.lda = ldy;
  g.B = W;
  g.ldb = ldw;
  g.M = (int)T;
  g.N = (int)k;
  g.K = (int)d;
  g.add = residual;
  g.ldadd = ldr;
  g.C = dX;
  g.ldc = ldx;
  return hip_status(logra::launch_gemm(logra::GemmForm::kInput, g, static_cast<char*>(ws), s));
}

int logra_linear_backward_weight(const uint16_t* dY, int64_t ldy, const uint16_t* X, int64_t ldx,
                                 int64_t T, int64_t d, int64_t k, int flags, void* dW, int dw_type,
                                 int64_t ldw, void* ws, size_t ws_bytes, hipStream_t s) {
  if (!sizes_ok(T, d, k) || !type_ok(dw_type)) return LOGRA_EINVAL;
  if ((flags & ~LOGRA_LINEAR_ACCUMULATE) != 0 || (flags != 0 && dw_type != LOGRA_F32))
    return LOGRA_EINVAL;
  if (!ld_ok(ldy, d, LOGRA_BF16) || !ld_ok(ldx, k, LOGRA_BF16) || !matrix_ok(dW, ldw, k, dw_type))
    return LOGRA_EINVAL;
  if (T == 0 && flags != 0) return LOGRA_OK;
  if (T > 0 && (!matrix_ok(dY, ldy, d, LOGRA_BF16) || !matrix_ok(X, ldx, k, LOGRA_BF16)))
    return LOGRA_EINVAL;
  if (!logra::gemm_fits(logra::GemmForm::kWeight, d, k, T)) return LOGRA_EINVAL;
  const size_t need = T > 0 ? logra::gemm_ws_bytes(logra::GemmForm::kWeight, d, k, T) : 0;
  if (!ws_ok(need, ws, ws_bytes)) return LOGRA_EWORKSPACE;
  const Span o = span(dW, d, k, ldw, bytes_of(dw_type));
  const Span w = span(need ? ws : nullptr, 1, (int64_t)need, 0, 1);
  const Span in[2] = {span(T > 0 ? dY : nullptr, T, d, ldy, 2),
                      span(T > 0 ? X : nullptr, T, k, ldx, 2)};
  if (any_overlap(o, in, 2) || any_overlap(w, in, 2) || overlap(o, w)) return LOGRA_EINVAL;
  logra::GemmArgs g{};
  g.A = dY;
  g.lda = ldy;
  g.B = X;
  g.ldb = ldx;
  g.M = (int)d;
  g.N = (int)k;
  g.K = (int)T;
  g.C = dW;
  g.ldc = ldw;
  g.c_f32 = dw_type == LOGRA_F32;
  g.accumulate = flags != 0;
  return hip_status(logra::launch_gemm(logra::GemmForm::kWeight, g, static_cast<char*>(ws), s));
}

}  // extern "C"
