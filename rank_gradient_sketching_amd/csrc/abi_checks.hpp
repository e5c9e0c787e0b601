// Argument checks that the C entry points of logra_policy.h and logra_step.h
// share (internal).
#pragma once

#include <math.h>
#include <stdint.h>

#include "logra_policy.h"

namespace logra {
namespace checks {

constexpr int64_t kDimLimit = int64_t(1) << 31;
constexpr int64_t kLdLimit = int64_t(1) << 40;

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}
inline bool dim_ok(int64_t x) { return x >= 1 && x < kDimLimit; }
inline bool type_ok(int t) { return t == LOGRA_BF16 || t == LOGRA_F32; }
inline int64_t bytes_of(int type) { return type == LOGRA_F32 ? 4 : 2; }
// 1 / tau and log2(e) / tau stay finite.
inline bool tau_ok(float tau) { return isfinite(tau) && tau > 0.0f && isfinite(1.5f / tau); }
// Row stride: >= row length, rows on 16-byte boundaries.
inline bool ld_ok(int64_t ld, int64_t row, int type) {
  return ld >= row && ld % (16 / bytes_of(type)) == 0 && ld < kLdLimit;
}

// Bytes [lo, hi) that a matrix of `rows` x `cols` elements spans.  One that passes
// the address space (strides reach 2^40) ends at kNoEnd and overlaps everything,
// which refuses it.
struct Span {
  uintptr_t lo, hi;
};
constexpr uintptr_t kNoEnd = ~uintptr_t(0);
inline Span span(const void* p, __int128 rows, __int128 cols, __int128 ld, int64_t elem) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  if (p == nullptr || rows == 0 || cols == 0) return Span{lo, lo};
  const __int128 hi = (__int128)lo + ((rows - 1) * ld + cols) * elem;
  return Span{lo, hi >= (__int128)kNoEnd ? kNoEnd : (uintptr_t)hi};
}
inline bool overlap(const Span& a, const Span& b) {
  if (a.hi == kNoEnd || b.hi == kNoEnd) return true;
  return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

}  // namespace checks
}  // namespace logra
