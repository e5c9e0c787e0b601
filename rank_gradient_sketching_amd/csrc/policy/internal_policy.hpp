// Host-side plans and kernel launchers of the policy-step operators
// (internal; the public boundary is include/logra_policy.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace logra {

// ---------------------------------------------------------------- log probabilities
constexpr int kMaxTop = 64;

// Tiling of a log-probability call: every row in n_split pieces of `piece`
// columns.  With more than one, each piece leaves its state (and its n_top
// best keys) in the workspace and a second kernel joins them.
struct LogprobPlan {
  int n_split;
  int64_t piece;
  size_t off_keys, total;   // workspace: float3 states, then 64-bit keys
};
LogprobPlan make_logprob_plan(int64_t n_tok, int64_t vocab, int n_top);

struct LogprobArgs {
  const void* z;
  int64_t ld;
  int64_t n_tok;
  int vocab;
  const int64_t* target;
  float tau;
  int n_top;
  float* logp;
  float* entropy;
  float* lse;
  int32_t* top_idx;
  float* top_logp;
};
hipError_t launch_token_logprob(const LogprobArgs& a, bool f32, const LogprobPlan& p, char* ws,
                                hipStream_t s);

struct LogprobGradArgs {
  const void* z;
  int64_t ld;
  int64_t n_tok;
  int vocab;
  const int64_t* target;
  float tau;
  const float* lse;
  const float* entropy;
  const float* d_logp;
  const float* d_entropy;
  const float* d_lse;
  void* dz;
  int64_t ldz;
};
hipError_t launch_token_logprob_backward(const LogprobGradArgs& a, bool f32, hipStream_t s);

// ---------------------------------------------------------------- AdamW
constexpr int kStateBlock = 32;
// The dither of the 8-bit states counts in two odd constants modulo 2^32, along
// the entries and along the steps: equally spaced values in any run of either.
constexpr uint32_t kDitherIndex = 0x6A09E667u;   // 2^32 times frac(sqrt 2)
constexpr uint32_t kDitherStep = 0x9E3779B9u;    // 2^32 times frac(golden ratio)

struct AdamwItem {
  void* p;
  const void* g;
  float* master;
  void* m;
  void* v;
  uint8_t* m_exp;
  uint8_t* v_exp;
  int64_t n;
  float weight_decay;
  uint32_t dither0;   // counter of the tensor's first entry
  int32_t vec;        // every array on a boundary of whole vectors
  int32_t pad;
};
struct AdamwScalars {
  float lr, b1, b2, c1, c2, eps;   // c = 1 - beta
  float inv_bc1, inv_sqrt_bc2;     // 1 / b1, 1 / sqrt(b2) (bias corrections)
  uint32_t dither_step;
  const float* grad_scale;
};
enum class AdamwWeights { kF32, kBf16, kBf16Master };
// The tensors of one form (weights, gradient type, state type) in a table: n
// items and their first work-groups, of `steps` steps each.
struct AdamwForm {
  int32_t n, groups, steps;
  uint32_t off_items, off_first;   // bytes from the table's start
};
constexpr int kAdamwForms = 12;
struct AdamwTable {
  uint64_t magic;
  uint64_t bytes;
  AdamwForm form[kAdamwForms];   // weights * 4 + fp32 gradient * 2 + 8-bit states
};
// Fills in a form's steps, groups, first work-groups and the items' vec (n and
// the items are set); false where the work-groups do not fit a launch.
bool adamw_lay_out(AdamwForm* form, AdamwItem* items, int32_t* first, bool g_f32, bool state8,
                   AdamwWeights weights);
hipError_t launch_adamw(AdamwWeights weights, bool g_f32, bool state8, const AdamwForm& form,
                        const AdamwItem* items, const int32_t* first, const AdamwScalars& h,
                        hipStream_t s);
hipError_t launch_adamw_state_values(bool second, const uint8_t* codes, const uint8_t* exps,
                                     int64_t n, uint16_t* out, hipStream_t s);

// ---------------------------------------------------------------- unmerged updates
struct AdapterPlan {
  int rp;            // r rounded up to 16, 32, 64, 128 or 256
  int n_split;       // pieces of k
  int chunks_per_split;   // 256-column chunks in one piece
  size_t total;      // workspace: fp32 P, [n_split][T][rp]
};
bool make_adapter_plan(int64_t T, int64_t d, int64_t k, int r, AdapterPlan* p);

struct AdapterArgs {
  const uint16_t* X;
  int64_t ldx;
  const uint16_t* Y;
  int64_t ldy;
  uint16_t* out;
  int64_t ldo;
  int64_t T;
  int d, k, r;
  int64_t n;
  const int32_t* adapter;
  const void* U;
  const uint64_t* seeds;
  const uint16_t* A;
  int64_t lda;
  const float* scale;
};
hipError_t launch_adapter(const AdapterArgs& a, bool u_f32, const AdapterPlan& p, char* ws,
                          hipStream_t s);

}  // namespace logra
