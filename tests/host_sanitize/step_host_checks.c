/* Host-side checks of logra_step.h, built with AddressSanitizer and
 * UndefinedBehaviorSanitizer.  Every call made here is rejected by the argument
 * checks before the first HIP call, or is a pure host function (workspace
 * sizes, the table of a gradient norm).  Device pointers are stand-in addresses
 * that are never dereferenced.
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "logra_step.h"

static int g_fail = 0;
static int g_checks = 0;

#define EXPECT(cond)                                                   \
  do {                                                                 \
    ++g_checks;                                                        \
    if (!(cond)) {                                                     \
      ++g_fail;                                                        \
      fprintf(stderr, "%s:%d: expectation failed: %s\n", __FILE__,     \
              __LINE__, #cond);                                        \
    }                                                                  \
  } while (0)

static void* at(int i) { return (void*)((uintptr_t)(i + 1) << 40); }

static const int64_t kDims[] = {INT64_MIN, -1, 0, 1, 2, 15, 16, 17, 255, 257, 8960, 152064,
                                (int64_t)1 << 20, (int64_t)1 << 28, ((int64_t)1 << 31) - 1,
                                (int64_t)1 << 31, INT64_MAX};
static const int64_t kLds[] = {INT64_MIN, 0, 8, 9, 256, (int64_t)1 << 39, ((int64_t)1 << 40) - 8,
                               (int64_t)1 << 40, INT64_MAX};
#define N_OF(a) ((int)(sizeof(a) / sizeof((a)[0])))

static int size_ok(int64_t x) { return x >= 1 && x < (int64_t)1 << 31; }

static void check_sizes(void) {
  for (int i = 0; i < N_OF(kDims); ++i)
    for (int j = 0; j < N_OF(kDims); ++j) {
      const size_t w = logra_sample_tokens_ws_bytes(kDims[i], kDims[j]);
      const size_t b = logra_linear_backward_act_ws_bytes(kDims[i], kDims[j]);
      EXPECT(w % 256 == 0 && b % 256 == 0);
      if (!size_ok(kDims[i]) || !size_ok(kDims[j])) EXPECT(w == 0);
      if (!size_ok(kDims[j])) EXPECT(b == 0);
      for (int k = 0; k < N_OF(kDims); ++k) {
        const size_t g = logra_linear_ws_bytes(kDims[i], kDims[j], kDims[k]);
        EXPECT(g % 256 == 0);
        if (!size_ok(kDims[i]) || !size_ok(kDims[j]) || !size_ok(kDims[k])) EXPECT(g == 0);
      }
    }
}

/* Sizes and strides of every magnitude, with an output over an input: nothing is
 * accepted but a batch without rows. */
static void check_calls(void) {
  const uint16_t *X = at(0), *W = at(1);
  for (int i = 0; i < N_OF(kDims); ++i)
    for (int j = 0; j < N_OF(kDims); ++j)
      for (int l = 0; l < N_OF(kLds); ++l) {
        const int64_t n = kDims[i], v = kDims[j], ld = kLds[l];
        if (n == 0) continue;
        const int st = logra_sample_tokens(at(0), LOGRA_BF16, n, v, ld, at(1), 1.0f, 4, 0.5f, 0.0f,
                                           NULL, NULL, NULL, NULL, at(0), at(2), at(3), at(4),
                                           at(5), SIZE_MAX, NULL);
        EXPECT(st == LOGRA_EINVAL);      /* the tokens lie over the logits */
        EXPECT(logra_sample_tokens(at(0), LOGRA_F32, n, v, ld, at(1), NAN, 0, 1.0f, 0.0f, NULL,
                                   NULL, NULL, NULL, at(2), NULL, NULL, NULL, at(5), SIZE_MAX,
                                   NULL) == LOGRA_EINVAL);
        EXPECT(logra_linear_backward_act(at(0), LOGRA_F32, ld, NULL, 0, LOGRA_ACT_NONE, n, v, at(0),
                                         ld, at(2), at(3), SIZE_MAX, NULL) == LOGRA_EINVAL);
        for (int k = 0; k < N_OF(kDims); ++k) {
          const int64_t c = kDims[k];
          EXPECT(logra_linear(X, ld, W, ld, n, v, c, NULL, 0, LOGRA_ACT_SILU, NULL, 0, at(0),
                              LOGRA_BF16, ld, NULL, 0, at(3), SIZE_MAX, NULL) == LOGRA_EINVAL);
          EXPECT(logra_linear_backward_input(X, ld, W, ld, n, v, c, NULL, 0, at(1), ld, at(3),
                                             SIZE_MAX, NULL) == LOGRA_EINVAL);
          EXPECT(logra_linear_backward_weight(X, ld, W, ld, n, v, c, 0, at(1), LOGRA_F32, ld,
                                              at(3), SIZE_MAX, NULL) == LOGRA_EINVAL);
        }
      }
}

/* Tables of up to a few thousand tensors in every form, in buffers of exactly
 * the size asked for. */
static void check_tables(void) {
  const int counts[] = {0, 1, 2, 63, 64, 65, 2000};
  for (int c = 0; c < N_OF(counts); ++c) {
    const int n = counts[c];
    logra_grad_item* items = (logra_grad_item*)calloc((size_t)n + 1, sizeof(*items));
    for (int i = 0; i < n; ++i) {
      items[i].g = at(0);
      items[i].g_type = i % 2;
      if (i % 3 == 0) {
        items[i].out = at(1);
        items[i].out_type = (i / 3) % 2;
      }
      items[i].n = i % 7 == 0 ? 0 : i % 11 == 0 ? ((int64_t)1 << 24) + i : 1000 + 37 * i;
    }
    const size_t bytes = logra_grad_table_bytes(n);
    char* table = (char*)malloc(bytes);
    EXPECT(logra_grad_table(n, items, table, bytes) == LOGRA_OK);
    EXPECT(logra_grad_table(n, items, table, bytes - 1) == LOGRA_EWORKSPACE);
    const size_t need = logra_grad_norm_ws_bytes(table);
    EXPECT(need >= 256 && need % 256 == 0);
    EXPECT(logra_grad_norm(table, NULL, LOGRA_NORM_2, NAN, NULL, at(2), at(3), NULL, at(4), need,
                           NULL) == LOGRA_EINVAL);
    EXPECT(logra_grad_norm(table, at(5), LOGRA_NORM_2, 1.0, NULL, at(2), at(3), NULL, at(4),
                           need - 1, NULL) == LOGRA_EWORKSPACE);
    EXPECT(logra_grad_clip(table, NULL, at(3), NULL) == (n > 1 ? LOGRA_EINVAL : LOGRA_OK));
    for (int i = 0; i < n; ++i) items[i].n = ((int64_t)1 << 40) - 1;   /* as large as can be */
    const int st = logra_grad_table(n, items, table, bytes);
    EXPECT(st == LOGRA_OK || st == LOGRA_EINVAL);
    EXPECT(logra_grad_norm_ws_bytes(table) % 256 == 0);
    free(table);
    free(items);
  }
  EXPECT(logra_grad_table_bytes(INT32_MIN) == 0 && logra_grad_table_bytes(INT32_MAX) == 0);
}

int main(void) {
  check_sizes();
  check_calls();
  check_tables();
  printf("%d checks, %d failed\n", g_checks, g_fail);
  return g_fail != 0;
}
