/* Host-side checks of logra_policy.h, built with AddressSanitizer and
 * UndefinedBehaviorSanitizer.  Every call made here is rejected by the argument
 * checks before the first HIP call, or is a pure host function (workspace
 * sizes, the table of an AdamW step).  Device pointers are stand-in addresses
 * that are never dereferenced.
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "logra_policy.h"

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

static const int64_t kDims[] = {-1, 0, 1, 2, 7, 8, 31, 32, 33, 255, 256, 257, 8960, 152064,
                                (int64_t)1 << 20, (int64_t)1 << 28, ((int64_t)1 << 31) - 1,
                                (int64_t)1 << 31, INT64_MAX, INT64_MIN};
static const int32_t kRanks[] = {INT32_MIN, -1, 0, 1, 16, 17, 64, 100, 255, 256, 257, INT32_MAX};
static const int64_t kLds[] = {INT64_MIN, 0, 8, 9, 256, (int64_t)1 << 39, ((int64_t)1 << 40) - 8,
                               (int64_t)1 << 40, INT64_MAX};
#define N_OF(a) ((int)(sizeof(a) / sizeof((a)[0])))

static void check_sizes(void) {
  for (int i = 0; i < N_OF(kDims); ++i)
    for (int j = 0; j < N_OF(kDims); ++j)
      for (int r = 0; r < N_OF(kRanks); ++r) {
        const size_t w = logra_token_logprob_ws_bytes(kDims[i], kDims[j], kRanks[r]);
        EXPECT(w % 256 == 0);
        for (int k = 0; k < N_OF(kDims); ++k) {
          const size_t b = logra_adapter_ws_bytes(kDims[i], kDims[j], kDims[k], kRanks[r]);
          EXPECT(b % 256 == 0);
          if (kRanks[r] < 1 || kRanks[r] > 256 || kDims[i] < 1 || kDims[j] < 1 || kDims[k] < 1)
            EXPECT(b == 0);
        }
      }
}

/* Sizes and strides of every magnitude: no workspace is given, so that nothing
 * is accepted; the gradient's rows pass the address space. */
static void check_calls(void) {
  for (int i = 0; i < N_OF(kDims); ++i)
    for (int j = 0; j < N_OF(kDims); ++j)
      for (int l = 0; l < N_OF(kLds); ++l) {
        const int64_t n = kDims[i], v = kDims[j], ld = kLds[l];
        if (n == 0) continue;
        EXPECT(logra_token_logprob(at(0), LOGRA_BF16, n, v, ld, at(1), 0.0f, 4, at(2), at(3),
                                   at(4), at(5), at(6), NULL, 0, NULL) == LOGRA_EINVAL);
        const int st = logra_token_logprob(at(0), LOGRA_F32, n, v, ld, at(1), 1.0f, 0, at(0),
                                           at(3), at(4), NULL, NULL, at(7), SIZE_MAX, NULL);
        EXPECT(st == LOGRA_EINVAL);     /* logp lies over the logits */
        EXPECT(logra_token_logprob_backward(at(0), LOGRA_BF16, n, v, ld, at(1), 1.0f, at(2), NULL,
                                            at(3), NULL, NULL, at(2), ld, NULL) == LOGRA_EINVAL);
        for (int r = 0; r < N_OF(kRanks); ++r) {
          EXPECT(logra_adapter_apply(at(0), ld, at(1), ld, at(2), ld, n, v, kDims[N_OF(kDims) - 1 - j],
                                     kRanks[r], n, at(3), at(4), LOGRA_F32, at(5), NULL, 0, at(6),
                                     NULL, 0, NULL) != LOGRA_OK);
          EXPECT(logra_adapter_apply(at(0), ld, at(1), ld, at(2), ld, n, v, v, kRanks[r], n, at(2),
                                     at(4), LOGRA_F32, NULL, at(5), ld, at(6), at(7), SIZE_MAX,
                                     NULL) == LOGRA_EINVAL);   /* the ids lie under out */
        }
      }
  EXPECT(logra_adamw_state_values(LOGRA_STATE_M, at(0), at(1), INT64_MAX, at(2), NULL) ==
         LOGRA_EINVAL);
  EXPECT(logra_adamw_state_values(LOGRA_STATE_V, at(0), at(1), ((int64_t)1 << 40) - 1, at(1),
                                  NULL) == LOGRA_EINVAL);
}

/* Tables of up to a few thousand tensors in every form, in buffers of exactly
 * the size asked for. */
static void check_tables(void) {
  const int counts[] = {0, 1, 2, 63, 64, 65, 2000};
  for (int c = 0; c < N_OF(counts); ++c) {
    const int n = counts[c];
    logra_adamw_item* items = (logra_adamw_item*)calloc((size_t)n + 1, sizeof(*items));
    for (int i = 0; i < n; ++i) {
      items[i].p = at(0);
      items[i].g = at(1);
      items[i].m = at(2);
      items[i].v = at(3);
      items[i].p_type = (i / 2) % 2;
      items[i].g_type = i % 2;
      if (i % 3 == 0) items[i].m_exp = items[i].v_exp = (uint8_t*)at(4);
      if (i % 5 == 0 && items[i].p_type == LOGRA_BF16) items[i].master = (float*)at(5);
      items[i].n = i % 7 == 0 ? 0 : i % 11 == 0 ? ((int64_t)1 << 24) + i : 1000 + 37 * i;
    }
    const size_t bytes = logra_adamw_table_bytes(n);
    char* table = (char*)malloc(bytes);
    EXPECT(logra_adamw_table(n, items, table, bytes) == LOGRA_OK);
    EXPECT(logra_adamw_table(n, items, table, bytes - 1) == LOGRA_EWORKSPACE);
    /* scalars that are refused, and the missing device copy where there is work */
    EXPECT(logra_adamw_step(table, NULL, NAN, 0.9, 0.99, 1e-8, 1, NULL, NULL) == LOGRA_EINVAL);
    EXPECT(logra_adamw_step(table, NULL, 1e-3, 0.9, 1.0, 1e-8, 1, NULL, NULL) == LOGRA_EINVAL);
    EXPECT(logra_adamw_step(table, NULL, 1e-3, 0.9, 0.99, 1e-8, INT64_MIN, NULL, NULL) ==
           LOGRA_EINVAL);
    EXPECT(logra_adamw_step(table, NULL, 1e-3, 0.9, 0.99, 1e-8, INT64_MAX, NULL, NULL) ==
           (n > 1 ? LOGRA_EINVAL : LOGRA_OK));
    if (n) {
      items[n - 1].n = ((int64_t)1 << 40) - 1;     /* more work-groups than a launch takes */
      EXPECT(logra_adamw_table(n, items, table, bytes) == LOGRA_EINVAL);
      EXPECT(logra_adamw_step(table, table, 1e-3, 0.9, 0.99, 1e-8, 1, NULL, NULL) == LOGRA_EINVAL);
    }
    free(table);
    free(items);
  }
  EXPECT(logra_adamw_table_bytes(INT32_MIN) == 0 && logra_adamw_table_bytes(INT32_MAX) == 0);
  EXPECT(logra_adamw_table_bytes(1 << 24) > 0);
}

int main(void) {
  check_sizes();
  check_calls();
  check_tables();
  printf("%d checks, %d failed\n", g_checks, g_fail);
  return g_fail != 0;
}
