// Host-side plans and kernel launchers of the operators that close a policy
// step (internal; the public boundary is include/logra_step.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace logra {

// ---------------------------------------------------------------- sampling
struct SampleArgs {
  const void* z;
  int64_t ld;
  int64_t n_tok;
  int vocab;
  const float* u;
  float tau;
  int32_t top_k;
  float top_p, min_p;
  const float* tau_rows;
  const int32_t* top_k_rows;
  const float* top_p_rows;
  const float* min_p_rows;
  int64_t* token;
  float* logp;
  float* logq;
  int32_t* kept;
};
size_t sample_ws_bytes(int64_t n_tok, int64_t vocab);
hipError_t launch_sample(const SampleArgs& a, bool f32, char* ws, hipStream_t s);

// ---------------------------------------------------------------- gradient norm
struct GradItem {
  void* g;
  void* out;
  int64_t n;
  int32_t g_f32, out_f32;
  int32_t vec;        // g and out on 16-byte boundaries
  int32_t pad;
};
// Head of a table; the items follow, then n + 1 first work-groups.
struct GradTable {
  uint64_t magic;
  uint64_t bytes;
  int32_t n, groups;
  int32_t loops;      // steps of a work-group
  int32_t large;      // more gradients than are worth keeping in the caches
};
// Fills in the head's loops, groups and large, the items' vec and the first work-groups;
// false where the work-groups do not fit a launch.
bool grad_lay_out(GradTable* head, GradItem* items, int32_t* first);
struct GradNormArgs {
  const GradItem* items;     // device
  const int32_t* first;      // device, n + 1
  int32_t n, groups, loops;
  bool large, inf_norm;
  double max_norm;
  const float* grad_scale;
  float* norm;
  float* scale;
  float* norms;
};
hipError_t launch_grad_norm(const GradNormArgs& a, double* partial, hipStream_t s);
hipError_t launch_grad_clip(const GradNormArgs& a, const float* scale, hipStream_t s);

// ---------------------------------------------------------------- layer product
enum Act { kActNone, kActRelu, kActSilu, kActGelu, kActGeluTanh, kActs };

// C[M x N] = sum over K of A(m, k) B(n, k), with an epilogue.  An operand is a
// matrix with rows along m (or n) and K contiguous, or the other way round
// (`along_k` rows: row k holds the operand's m or n contiguously).
struct GemmArgs {
  const uint16_t* A;
  int64_t lda;
  const uint16_t* B;
  int64_t ldb;
  int M, N, K;
  const void* bias;       // per column n, or null
  bool bias_f32;
  int act;
  const uint16_t* add;    // bf16 [M x ldadd], or null
  int64_t ldadd;
  void* C;
  int64_t ldc;
  bool c_f32, accumulate;
  uint16_t* pre;          // bf16 [M x ldpre], or null
  int64_t ldpre;
};
enum class GemmForm { kForward, kInput, kWeight };   // A, B along k: neither; B; both
// Whether a product fits a launch.
bool gemm_fits(GemmForm form, int64_t M, int64_t N, int64_t K);
size_t gemm_ws_bytes(GemmForm form, int64_t M, int64_t N, int64_t K);
hipError_t launch_gemm(GemmForm form, const GemmArgs& a, char* ws, hipStream_t s);

struct ActGradArgs {
  const void* d_out;
  bool d_out_f32;
  int64_t ldd;
  const uint16_t* pre;
  int64_t ldp;
  int act;
  int64_t T;
  int d;
  uint16_t* dY;
  int64_t ldy;
  float* d_bias;
};
size_t act_grad_ws_bytes(int64_t T, int64_t d);
hipError_t launch_act_grad(const ActGradArgs& a, char* ws, hipStream_t s);

}  // namespace logra
