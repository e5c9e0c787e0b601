// logra_token_logprob and its gradient, on gfx950: log probabilities of given
// tokens under softmax(z / tau), the entropy of that distribution and its most
// probable tokens, in one pass over the logits.
//
// Mathematics.  With a reference logit m of the row, d_j = (z_j - m) log2(e) / tau
// and w_j = 2^d_j, a row needs s = sum w and u = sum w d:
//   lse = m / tau + ln s,   logp = ln(2) d_target - ln s,
//   H = ln s - ln(2) u / s.
// None of the three depends on m, which need only be near enough to the largest
// logit that no weight overflows: a thread keeps the largest of the group that
// set it and looks at its elements' maximum again only when a group's weights
// sum to more than 2^10.  d is one fused step, z l2t - mc with l2t = log2(e) /
// tau and mc = m l2t rounded: that rounding is the same for every token of the
// row, cancels in logp and H, and is added back in lse, so rows far from zero
// keep their accuracy.  It stays a small one (half a binade of a weight) only up to
// |m l2t| = 2^24; past that (rows masked with -1e30, or at the type's lowest value)
// mc is held as infinite, the fused step fails for every group, and the careful path
// takes the difference z - m first, which is exact wherever its weight is not zero.
// That path also takes the groups with a masked token (z = -inf: w = 0, d clamped
// at kLow in u, so that 0 * -inf does not arise); NaN, and +inf, which becomes NaN,
// still reach s.
// The states of a wave meet in a butterfly and those of a row's waves in LDS,
// always in the same order.
// Alternatives.  Value and index of a token make one 64-bit key (the float's
// bits in an order-preserving form above the inverted index), so "larger logit,
// then lower index" is one integer comparison and keys are distinct: the result
// does not depend on the order of anything.  What the stream keeps are not tokens
// but runs of neighbours (a lane's 16 bytes), keyed by their largest logit: the
// n_top best runs hold the n_top best tokens, because each run before a token's
// own has a better one.  A run whose largest logit (one comparison) does not beat
// the n_top-th so far is dropped; others wait in LDS, and 64 of them at a time are
// sorted by a bitonic network and merged in.  On a wave's first group the lanes'
// maxima alone are sorted (32-bit values): their n_top-th is a threshold that most
// other runs fail, so that usually all of a work-group's keys fit one sort at the
// end.  The best runs' tokens are then read again and sorted.
//
// Bound: the stream of the logits and, close behind it, the vector unit (eight
// elements cost about 70 issue slots, 32 of them the exponentials).  One
// work-group per row where the rows fill the chip; fewer rows are cut into pieces
// whose states and keys a second kernel joins.  4096 x 152064 bf16: 199 us, 6.3
// TB/s.  8 rows of it with eight alternatives: 8.9 + 6.7 us (5.4 + 3.3 without),
// 501 x 32003 fp32 with five 23.3 + 5.5 (16.7 + 3.9 without).
#include <math.h>

#include "common.hpp"
#include "internal.hpp"
#include "policy/internal_policy.hpp"

namespace logra {

namespace {

typedef unsigned long long u64;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLow = -1000.0f;   // 2^kLow is 0 in fp32
constexpr float kLowLn = -128.0f;  // and so is e^kLowLn
constexpr float kMinFloat = -3.4028234663852886e38f;
constexpr float kFusedEnd = 0x1p24f;   // half a step of fp32 below it is at most 1/2

// ---------------------------------------------------------------- softmax states
struct State {
  float m, s, u;
};

// The rounded product m l2t of a reference that the fused step may be taken about;
// infinite for others.
__device__ __forceinline__ float centre(float m, float l2t) {
  const float c = m * l2t;
  return fabsf(c) < kFusedEnd ? c : INFINITY;
}
// d of logit z about the reference m, mc = centre(m, l2t).
__device__ __forceinline__ float exponent(float z, float m, float mc, float l2t) {
  return isfinite(mc) ? fmaf(z, l2t, -mc) : (z - m) * l2t;
}
// The reference a as seen from the reference M >= a, clamped (ca, cM: their
// centres): a difference of what the weights were formed about, the rounded product
// (so that nothing may be fused into it) or, past the fused step's end, the exact one.
__device__ __forceinline__ float shift(float a, float ca, float M, float cM, float l2t) {
#pragma clang fp contract(off)
  float d = ca - cM;
  if (__builtin_expect(!isfinite(d), 0))
    d = isfinite(ca) ? fmaf(-M, l2t, ca) : isfinite(cM) ? fmaf(a, l2t, -cM) : (a - M) * l2t;
  return fmaxf(d, kLow);
}

__device__ __forceinline__ State merge_states(const State& a, const State& b, float l2t) {
  // about the larger reference, so that only the other one moves
  const bool up = b.m > a.m;
  const State hi{up ? b.m : a.m, up ? b.s : a.s, up ? b.u : a.u};
  const State lo{up ? a.m : b.m, up ? a.s : b.s, up ? a.u : b.u};
  const float d = shift(lo.m, centre(lo.m, l2t), hi.m, centre(hi.m, l2t), l2t);
  const float f = exp2_normal(d);
  return State{hi.m, fmaf(f, lo.s, hi.s), fmaf(f, fmaf(lo.s, d, lo.u), hi.u)};
}

__device__ __forceinline__ State wave_state(State st, float l2t) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    State o;
    o.m = __shfl_xor(st.m, off);
    o.s = __shfl_xor(st.s, off);
    o.u = __shfl_xor(st.u, off);
    st = merge_states(st, o, l2t);
  }
  return st;
}

// Adds G elements; mc = centre(st.m, l2t) goes along.
template <int G>
__device__ __forceinline__ void add_group(State& st, float& mc, const float* z, float l2t) {
  float gs, gu;
#pragma unroll
  for (int e = 0; e < G; ++e) {
    const float d = fmaf(z[e], l2t, -mc);
    const float w = exp2_normal(d);
    gs = e ? gs + w : w;
    gu = e ? fmaf(w, d, gu) : w * d;
  }
  // (2^10: the reference stays near enough for H to lose no more than ln 2^10
  // roundings where ln s and u / s nearly cancel)
  const bool careful = !(gs <= 0x1p10f) || gu != gu;
  if (__builtin_expect(__ballot(careful) != 0, 0) && careful) {
    float gmax = z[0];
#pragma unroll
    for (int e = 1; e < G; ++e) gmax = fmaxf(gmax, z[e]);
    if (gmax > st.m) {
      const float c = centre(gmax, l2t);
      const float dm = shift(st.m, mc, gmax, c, l2t);
      const float f = exp2_normal(dm);
      st.u = f * fmaf(st.s, dm, st.u);
      st.s *= f;
      st.m = gmax;
      mc = c;
    }
    gs = gu = 0.0f;
#pragma unroll
    for (int e = 0; e < G; ++e) {
      const float d = exponent(z[e], st.m, mc, l2t);
      const float w = exp2_normal(d);
      gs += w;
      gu = fmaf(w, fmaxf(d, kLow), gu);
    }
  }
  st.s += gs;
  st.u += gu;
}

// ---------------------------------------------------------------- best keys
__device__ __forceinline__ u64 order_key(float x, uint32_t idx) {
  uint32_t b = __float_as_uint(x + 0.0f);   // (-0 orders as +0)
  b ^= (uint32_t)((int32_t)b >> 31) | 0x80000000u;
  return ((u64)b << 32) | (0xFFFFFFFFu - idx);
}
__device__ __forceinline__ float key_value(u64 key) {
  const uint32_t b = (uint32_t)(key >> 32);
  return __uint_as_float((b & 0x80000000u) ? b ^ 0x80000000u : ~b);
}
__device__ __forceinline__ int key_index(u64 key) { return (int)(0xFFFFFFFFu - (uint32_t)key); }

// The key of lane l ^ J, by moves inside the vector unit (a __shfl_xor goes
// through LDS; the sorts below are chains of these): J = 1, 2 permute a quad;
// reversing 8 lanes (l ^ 7) and then each quad (l ^ 3) is l ^ 4, reversing 16 and
// then 8 is l ^ 8; 16 and 32 swap row pairs and wave halves.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true);
}
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E, kQuadXor3 = 0x1B;   // quad_perm
constexpr int kMirror8 = 0x141, kMirror16 = 0x140;                    // row_half_mirror, row_mirror
template <int J>
__device__ __forceinline__ uint32_t lane_xor(uint32_t x) {
  if constexpr (J == 1) {
    return dpp<kQuadXor1>(x);
  } else if constexpr (J == 2) {
    return dpp<kQuadXor2>(x);
  } else if constexpr (J == 4) {
    return dpp<kQuadXor3>(dpp<kMirror8>(x));
  } else if constexpr (J == 8) {
    return dpp<kMirror8>(dpp<kMirror16>(x));
  } else if constexpr (J == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return (threadIdx.x & 16) ? r[0] : r[1];
  } else {
    return swap_halves(x);
  }
}
template <int J>
__device__ __forceinline__ u64 compare_exchange(u64 x, bool keep_max) {
  const u64 y = ((u64)lane_xor<J>((uint32_t)(x >> 32)) << 32) | lane_xor<J>((uint32_t)x);
  return (x > y) == keep_max ? x : y;
}
template <int J>
__device__ __forceinline__ uint32_t compare_exchange(uint32_t x, bool keep_max) {
  const uint32_t y = lane_xor<J>(x);
  return keep_max ? max(x, y) : min(x, y);
}
// One bitonic merge of runs of K lanes, descending where `down`.
template <int K, class Key>
__device__ __forceinline__ Key bitonic(Key x, bool down) {
  const int lane = threadIdx.x & 63;
  if constexpr (K >= 64) x = compare_exchange<32>(x, ((lane & 32) == 0) == down);
  if constexpr (K >= 32) x = compare_exchange<16>(x, ((lane & 16) == 0) == down);
  if constexpr (K >= 16) x = compare_exchange<8>(x, ((lane & 8) == 0) == down);
  if constexpr (K >= 8) x = compare_exchange<4>(x, ((lane & 4) == 0) == down);
  if constexpr (K >= 4) x = compare_exchange<2>(x, ((lane & 2) == 0) == down);
  return compare_exchange<1>(x, ((lane & 1) == 0) == down);
}
// Sorted over the wave's lanes, descending where `down`.
template <class Key>
__device__ __forceinline__ Key sort_lanes(Key x, bool down) {
  const int lane = threadIdx.x & 63;
  x = bitonic<2>(x, ((lane & 2) != 0) != down);
  x = bitonic<4>(x, ((lane & 4) != 0) != down);
  x = bitonic<8>(x, ((lane & 8) != 0) != down);
  x = bitonic<16>(x, ((lane & 16) != 0) != down);
  x = bitonic<32>(x, ((lane & 32) != 0) != down);
  return bitonic<64>(x, down);
}

// Places for keys that wait: fewer than 64, and two runs of every lane.
constexpr int kBuf = 64 + 64 * 2;

// Keys of a wave that may be among the n_top best of its elements: some wait,
// unsorted, in LDS; once 64 do they are merged into a sorted list of 64 (lane i
// the i-th best, 0: none).
struct BestKeys {
  u64 best;
  u64 thr_key;   // a key below which nothing is among the n_top best
  float thr;     // its value (-inf while there is none)
  int count;     // keys waiting in buf (below 64 between groups)
  bool merged;   // whether best holds any
  u64* buf;      // this wave's kBuf places in LDS
};

__device__ __forceinline__ BestKeys no_keys(u64* buf) {
  return BestKeys{0, 0, -INFINITY, 0, false, buf};
}

// Merges 64 more keys (0: none), ascending over the lanes.
__device__ __forceinline__ void merge_sorted(BestKeys& b, u64 x, int n_top) {
  // descending against ascending: the larger of each pair are the best 64
  b.best = bitonic<64>(b.best > x ? b.best : x, true);
  const uint32_t lo = __shfl((uint32_t)b.best, n_top - 1);
  const uint32_t hi = __shfl((uint32_t)(b.best >> 32), n_top - 1);
  const u64 key = ((u64)hi << 32) | lo;
  if (key > b.thr_key) {
    b.thr_key = key;
    b.thr = key_value(key);
  }
  b.merged = true;
}

// LDS writes of this wave's lanes before, their reads after.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Merges the keys that wait, 64 at a time from the end, until fewer than `keep`.
__device__ __forceinline__ void flush_keys(BestKeys& b, int keep, int n_top) {
  const int lane = threadIdx.x & 63;
  wave_sync();
#pragma unroll 1
  while (b.count >= keep) {
    const int at = b.count > 64 ? b.count - 64 : 0;
    const u64 x = at + lane < b.count ? b.buf[at + lane] : 0;
    b.count = at;
    if (__ballot(x > b.thr_key) != 0) merge_sorted(b, sort_lanes(x, false), n_top);
  }
  wave_sync();
}

// Lets one key per lane wait (every lane of the wave calls this).
__device__ __forceinline__ void append(BestKeys& b, u64 key, bool take) {
  const bool pass = take && key >= b.thr_key;
  const u64 mask = __ballot(pass);
  if (pass) b.buf[b.count + __popcll(mask & ((u64(1) << (threadIdx.x & 63)) - 1))] = key;
  b.count += __popcll(mask);
}

// A threshold from one value per lane (x: order-preserving bits, 0: none), each
// that of an element of its own: at least n_top elements are not below the
// n_top-th largest.
__device__ __forceinline__ void first_threshold(BestKeys& b, uint32_t x, int n_top) {
  const uint32_t v = __shfl(sort_lanes(x, true), n_top - 1);
  if (v != 0) {
    b.thr_key = (u64)v << 32;      // (any index)
    b.thr = key_value(b.thr_key);
  }
}

// The runs of a lane's group (GT::kRun neighbours each), keyed by their largest
// logit and first column.
template <class GT>
__device__ __forceinline__ void offer_group(BestKeys& b, const float* z, int64_t col, bool first,
                                            int n_top) {
  constexpr int kRuns = GT::G / GT::kRun;
  float top[kRuns];
  float gmax = -INFINITY;
#pragma unroll
  for (int i = 0; i < kRuns; ++i) {
    top[i] = z[GT::kRun * i];
#pragma unroll
    for (int e = 1; e < GT::kRun; ++e) top[i] = fmaxf(top[i], z[GT::kRun * i + e]);
    gmax = fmaxf(gmax, top[i]);
  }
  if (first)
    first_threshold(b, gmax > -INFINITY ? (uint32_t)(order_key(gmax, 0) >> 32) : 0, n_top);
  // Elements of later groups have larger indices than all before them, so an
  // equal value does not pass; inside a group the keys decide.
  if (__ballot(first ? gmax > -INFINITY : gmax > b.thr) == 0) return;
#pragma unroll
  for (int i = 0; i < kRuns; ++i)
    append(b, order_key(top[i], (uint32_t)GT::column(col, GT::kRun * i)),
           top[i] > -INFINITY && (first || top[i] > b.thr));
  if (b.count >= 64) flush_keys(b, 64, n_top);
}

// From the n_top best runs of a row (b.best) its n_top best tokens.
template <class GT, class T>
__device__ __forceinline__ void best_tokens(BestKeys& b, const T* z, int V, int n_top) {
  const int lane = threadIdx.x & 63;
  const u64 runs = b.best;
  const int n = __popcll(__ballot(lane < n_top && runs != 0));
  if (n * GT::kRun <= 64) {
    const uint32_t lo = __shfl((uint32_t)runs, lane / GT::kRun);
    const int64_t col = (int64_t)(0xFFFFFFFFu - lo) + lane % GT::kRun;
    const float x = lane < n * GT::kRun && col < V ? GT::one(z, col) : -INFINITY;
    b.best = sort_lanes(x > -INFINITY ? order_key(x, (uint32_t)col) : 0, true);
    return;
  }
  BestKeys t = no_keys(b.buf);
  // (n_top runs have a token not below the last one's best)
  if (n == n_top)
    t.thr_key = (u64)__shfl((uint32_t)(runs >> 32), n_top - 1) << 32;
  for (int i = 0; i < n * GT::kRun; i += 64) {
    const int r = (i + lane) / GT::kRun;
    const uint32_t lo = __shfl((uint32_t)runs, r & 63);
    const int64_t col = (int64_t)(0xFFFFFFFFu - lo) + (i + lane) % GT::kRun;
    const bool in = r < n && col < V;
    const float x = in ? GT::one(z, col) : -INFINITY;
    append(t, order_key(x, (uint32_t)col), x > -INFINITY);
    if (t.count >= 64) flush_keys(t, 64, n_top);
  }
  flush_keys(t, 1, n_top);
  b.best = t.best;
}

// ---------------------------------------------------------------- loads
// Eight elements of a lane: a wave covers 512 consecutive columns from `col` (the
// same in all of its lanes) with whole 16-byte loads.  bf16: one load, columns col
// + 8 lane + e.  fp32: two, columns col + 4 lane + e and 256 further.  load and
// store take the address of column col and a whole group; the tail forms take the
// row and stop at `end` (elements past it are -inf).
template <class T>
struct Group;
template <>
struct Group<uint16_t> {
  static constexpr int G = 8;
  static constexpr int kRun = 8;   // neighbouring columns
  struct Raw {
    u32x4 v;
  };
  static __device__ __forceinline__ int64_t column(int64_t col, int e) {
    return col + 8 * (int)(threadIdx.x & 63) + e;
  }
  static __device__ __forceinline__ Raw load(const uint16_t* at) {
    return Raw{__builtin_nontemporal_load(reinterpret_cast<const u32x4*>(at) + (threadIdx.x & 63))};
  }
  static __device__ __forceinline__ void values(const Raw& r, float* z) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      z[2 * p] = bf16_lo(r.v[p]);
      z[2 * p + 1] = bf16_hi(r.v[p]);
    }
  }
  static __device__ __forceinline__ void store(uint16_t* at, const float* z) {
    u32x4 v;
#pragma unroll
    for (int p = 0; p < 4; ++p) v[p] = pack_bf16x2(z[2 * p], z[2 * p + 1]);
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(at) + (threadIdx.x & 63));
  }
  static __device__ __forceinline__ float one(const uint16_t* row, int64_t col) {
    return bf16_to_f32(row[col]);
  }
  static __device__ __forceinline__ uint16_t of(float x) { return f32_to_bf16(x); }
};
template <>
struct Group<float> {
  static constexpr int G = 8;
  static constexpr int kRun = 4;
  struct Raw {
    f32x4 v[2];
  };
  static __device__ __forceinline__ int64_t column(int64_t col, int e) {
    return col + 4 * (int)(threadIdx.x & 63) + (e & 3) + 256 * (e >> 2);
  }
  static __device__ __forceinline__ Raw load(const float* at) {
    Raw r;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      r.v[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(at) + 64 * i +
                                          (threadIdx.x & 63));
    return r;
  }
  static __device__ __forceinline__ void values(const Raw& r, float* z) {
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = r.v[e >> 2][e & 3];
  }
  static __device__ __forceinline__ void store(float* at, const float* z) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x4 v = {z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]};
      __builtin_nontemporal_store(v, reinterpret_cast<f32x4*>(at) + 64 * i + (threadIdx.x & 63));
    }
  }
  static __device__ __forceinline__ float one(const float* row, int64_t col) { return row[col]; }
  static __device__ __forceinline__ float of(float x) { return x; }
};
template <class T>
__device__ __forceinline__ void load_tail(const T* row, int64_t col, int64_t end, float* z) {
  typedef Group<T> GT;
#pragma unroll
  for (int e = 0; e < GT::G; ++e) {
    const int64_t at = GT::column(col, e);
    z[e] = at < end ? GT::one(row, at) : -INFINITY;
  }
}
template <class T>
__device__ __forceinline__ void store_tail(T* row, int64_t col, int64_t end, const float* z) {
  typedef Group<T> GT;
#pragma unroll
  for (int e = 0; e < GT::G; ++e) {
    const int64_t at = GT::column(col, e);
    if (at < end) row[at] = GT::of(z[e]);
  }
}

constexpr int kWaveCols = 512;                    // columns of a wave's group
constexpr int64_t kStepCols = kWaves * kWaveCols;  // of a work-group's

// ---------------------------------------------------------------- results of a row
__device__ __forceinline__ bool left_out(const LogprobArgs& a, int64_t row) {
  if (a.target == nullptr) return false;
  const int64_t t = a.target[row];
  return t < 0 || t >= a.vocab;
}

// log p of logit z in a row with state st.  (In units of log2 a logit at the
// type's lowest value would overflow.)
__device__ __forceinline__ float log_p(float z, const State& st, float l2t, float tau) {
  const float d = kLn2 * exponent(z, st.m, centre(st.m, l2t), l2t);
  return (isfinite(d) ? d : (z - st.m) / tau) - logf(st.s);
}
// By one thread of the row.
__device__ __forceinline__ void write_row(const LogprobArgs& a, int64_t row, const State& st,
                                          float l2t, float zt) {
  const float ln_s = logf(st.s);
  const float mc = centre(st.m, l2t);
  if (a.lse) {
    // (the weights are off by the rounding of mc, all alike)
    const float off = isfinite(mc) ? kLn2 * fmaf(st.m, l2t, -mc) : 0.0f;
    a.lse[row] = st.m / a.tau + (ln_s - off);
  }
  if (a.entropy) a.entropy[row] = ln_s - kLn2 * (st.u / st.s);
  if (a.logp) a.logp[row] = log_p(zt, st, l2t, a.tau);
}
// The target's logit (0 where it is not asked for); the row is not left out.
template <class T>
__device__ __forceinline__ float target_logit(const LogprobArgs& a, int64_t row) {
  return a.logp ? Group<T>::one(static_cast<const T*>(a.z) + row * a.ld, a.target[row]) : 0.0f;
}
// By the lanes of one wave of the row.
__device__ __forceinline__ void write_keys(const LogprobArgs& a, int64_t row, const State& st,
                                           float l2t, u64 key) {
  const int lane = threadIdx.x & 63;
  if (lane >= a.n_top) return;
  a.top_idx[row * a.n_top + lane] = key ? key_index(key) : -1;
  a.top_logp[row * a.n_top + lane] = key ? log_p(key_value(key), st, l2t, a.tau) : -INFINITY;
}
__device__ __forceinline__ void write_left_out(const LogprobArgs& a, int64_t row) {
  if (threadIdx.x == 0) {
    if (a.logp) a.logp[row] = 0.0f;
    if (a.entropy) a.entropy[row] = 0.0f;
    if (a.lse) a.lse[row] = 0.0f;
  }
  if ((int)threadIdx.x < a.n_top) {
    a.top_idx[row * a.n_top + threadIdx.x] = -1;
    a.top_logp[row * a.n_top + threadIdx.x] = -INFINITY;
  }
}

// ---------------------------------------------------------------- kernels
// One task: columns [piece p, piece (p + 1)) of a row.  n_split == 1 writes the
// row's results; otherwise the piece's state and keys go to the workspace.
template <class T, bool TOP>
__global__ __launch_bounds__(kThreads) void logprob_rows_kernel(LogprobArgs a, int n_split,
                                                                int64_t piece,
                                                                float* __restrict__ states,
                                                                u64* __restrict__ keys) {
  typedef Group<T> GT;
  __shared__ State wst[kWaves];
  __shared__ int waiting[kWaves];
  __shared__ u64 wbuf[TOP ? kWaves * kBuf : 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const float l2t = kLog2e / a.tau;
  const int64_t n_tasks = a.n_tok * n_split;
  for (int64_t task = blockIdx.x; task < n_tasks; task += gridDim.x) {
    const int64_t row = task / n_split;
    const int sp = (int)(task - row * n_split);
    if (left_out(a, row)) {
      if (sp == 0) write_left_out(a, row);
      continue;
    }
    const T* z = static_cast<const T*>(a.z) + row * a.ld;
    const int64_t c0 = sp * piece;
    const int64_t c1 = c0 + piece < a.vocab ? c0 + piece : a.vocab;
    State st{kMinFloat, 0.0f, 0.0f};
    float mc = centre(st.m, l2t);
    BestKeys bk = no_keys(wbuf + (TOP ? wave * kBuf : 0));
    bool first = true;
    auto add = [&](const float* v, int64_t c) {
      add_group<GT::G>(st, mc, v, l2t);
      if constexpr (TOP) {
        offer_group<GT>(bk, v, c, first, a.n_top);
        first = false;
      }
    };
    // This wave's groups: whole ones, kDeep loaded ahead of their use (past the
    // last one it is loaded again, which spares the loop a condition), then what
    // is left of the piece.
    constexpr int kDeep = 2;
    int64_t c = c0 + wave * kWaveCols;
    const int64_t whole = c + kWaveCols <= c1 ? (c1 - kWaveCols - c) / kStepCols + 1 : 0;
    if (whole > 0) {
      const int64_t last = c + (whole - 1) * kStepCols;
      typename GT::Raw raw[kDeep];
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        const int64_t at = c + i * kStepCols;
        raw[i] = GT::load(z + (at < last ? at : last));
      }
      while (c <= last) {
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
          if (c > last) break;
          float v[GT::G];
          GT::values(raw[i], v);
          const int64_t at = c + kDeep * kStepCols;
          raw[i] = GT::load(z + (at < last ? at : last));
          add(v, c);
          c += kStepCols;
        }
      }
    }
    if (c < c1) {
      float v[GT::G];
      load_tail(z, c, c1, v);
      add(v, c);
    }
    st = wave_state(st, l2t);
    if (lane == 0) {
      wst[wave] = st;
      // (64 stands for more than fit one sort)
      if constexpr (TOP) waiting[wave] = bk.merged ? 64 : bk.count;
    }
    __syncthreads();
    bool few = true;
    if constexpr (TOP) {
      int total = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) total += waiting[w] + (waiting[w] >= 64 ? 64 : 0);
      few = total <= 64;
      if (!few) {
        flush_keys(bk, 1, a.n_top);
        wbuf[wave * kBuf + lane] = bk.best;
        __syncthreads();
      }
    }
    if (wave == 0) {
      State t = wst[0];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) t = merge_states(t, wst[w], l2t);
      if constexpr (TOP) {
        if (few) {
          // all waves' keys fit the lanes of one
          u64 x = 0;
          int at = lane;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) {
            if (at >= 0 && at < waiting[w]) x = wbuf[w * kBuf + at];
            at -= waiting[w];
          }
          bk.best = sort_lanes(x, true);
        } else {
#pragma unroll 1
          for (int w = 1; w < kWaves; ++w)
            merge_sorted(bk, wbuf[w * kBuf + 63 - lane], a.n_top);
        }
      }
      if (n_split == 1) {
        if (lane == 0) write_row(a, row, t, l2t, target_logit<T>(a, row));
        if constexpr (TOP) {
          best_tokens<GT>(bk, z, a.vocab, a.n_top);
          write_keys(a, row, t, l2t, bk.best);
        }
      } else {
        if (lane == 0) {
          states[3 * task] = t.m;
          states[3 * task + 1] = t.s;
          states[3 * task + 2] = t.u;
        }
        if constexpr (TOP) {
          if (lane < a.n_top) keys[task * a.n_top + lane] = bk.best;
        }
      }
    }
    __syncthreads();   // wst and wbuf are free for the next task
  }
}

// Joins the pieces of a row, one wave per row.
template <class T, bool TOP>
__global__ __launch_bounds__(64) void logprob_join_kernel(LogprobArgs a, int n_split,
                                                          const float* __restrict__ states,
                                                          const u64* __restrict__ keys) {
  __shared__ u64 buf[TOP ? kBuf : 1];
  const int lane = threadIdx.x;
  const float l2t = kLog2e / a.tau;
  for (int64_t row = blockIdx.x; row < a.n_tok; row += gridDim.x) {
    // (what the row needs is loaded at once, and keys that fit the lanes are sorted
    // as they are: 501 rows in 5.2 us, one after the other through LDS 6.5)
    const int64_t target = a.target ? a.target[row] : 0;
    State st{kMinFloat, 0.0f, 0.0f};
    const float* sq = states + 3 * row * n_split;
    if (lane < n_split) st = State{sq[3 * lane], sq[3 * lane + 1], sq[3 * lane + 2]};
    const int n = n_split * a.n_top;
    const u64* q = keys + row * n;
    u64 x0 = 0;
    // (more than fit the lanes: the pieces' best keys, for a threshold)
    if constexpr (TOP) {
      if (n <= 64)
        x0 = lane < n ? q[lane] : 0;
      else
        x0 = lane < n_split ? q[lane * a.n_top] : 0;
    }
    if (target < 0 || target >= a.vocab) continue;
    const float zt = target_logit<T>(a, row);
    for (int i = lane + 64; i < n_split; i += 64)
      st = merge_states(st, State{sq[3 * i], sq[3 * i + 1], sq[3 * i + 2]}, l2t);
    st = wave_state(st, l2t);
    if (lane == 0) write_row(a, row, st, l2t, zt);
    if constexpr (TOP) {
      BestKeys bk = no_keys(buf);
      if (n <= 64) {
        bk.best = sort_lanes(x0, true);
      } else {
        // the pieces' best keys first: their n_top-th leaves few others
        first_threshold(bk, (uint32_t)(x0 >> 32), a.n_top);
        constexpr int kAtOnce = 4;
        for (int i = 0; i < n; i += 64 * kAtOnce) {
          u64 x[kAtOnce];
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j)
            x[j] = i + 64 * j + lane < n ? q[i + 64 * j + lane] : 0;
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) {
            append(bk, x[j], x[j] != 0);
            if (bk.count >= 64) flush_keys(bk, 64, a.n_top);
          }
        }
        flush_keys(bk, 1, a.n_top);
      }
      best_tokens<Group<T>>(bk, static_cast<const T*>(a.z) + row * a.ld, a.vocab, a.n_top);
      write_keys(a, row, st, l2t, bk.best);
    }
  }
}

// dz over pieces of grad_groups groups per thread: 64 bytes of logits in flight
// per lane (4096 x 152064 bf16: 2, 4, 8 groups 417, 400, 428 us; 501 x 32003 fp32:
// 2, 4, 8 groups 23.0, 25.0, 28.2 us).
constexpr int grad_groups(size_t elem) { return elem == 2 ? 4 : 2; }
constexpr int64_t grad_cols(size_t elem) { return kStepCols * grad_groups(elem); }

template <class T>
__global__ __launch_bounds__(kThreads) void logprob_grad_kernel(LogprobGradArgs a, int n_pieces) {
  typedef Group<T> GT;
  constexpr int G = GT::G;
  constexpr int kGradGroups = grad_groups(sizeof(T));
  const int64_t n_tasks = a.n_tok * n_pieces;
  const int64_t V = a.vocab;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // 1 / tau as two floats: z / tau keeps fp32 accuracy in one fused step (a bf16
  // result has no use for it)
  const float ih = 1.0f / a.tau;
  const float il = fmaf(-a.tau, ih, 1.0f) / a.tau;
  // (below this z / tau is past fp32's range and il's part does not matter, but
  // would overflow by itself)
  const float z_low = kMinFloat * fminf(a.tau, 1.0f);
  for (int64_t task = blockIdx.x; task < n_tasks; task += gridDim.x) {
    const int64_t row = task / n_pieces;
    const int64_t c0 = (task - row * n_pieces) * grad_cols(sizeof(T)) + wave * kWaveCols;
    const T* z = static_cast<const T*>(a.z) + row * a.ld;
    T* dz = static_cast<T*>(a.dz) + row * a.ldz;
    const int64_t target = a.target ? a.target[row] : -1;
    const bool out = a.target && (target < 0 || target >= V);
    const float lse = a.lse[row];
    const float g = a.d_logp ? a.d_logp[row] : 0.0f;
    const float gl = a.d_lse ? a.d_lse[row] : 0.0f;
    const float gh = a.d_entropy ? a.d_entropy[row] : 0.0f;
    const float H = a.d_entropy ? a.entropy[row] : 0.0f;
    // dz_j = p_j (k0 + k1 log p_j) + [j = target] kt
    // (lse - lse: NaN where it is not finite, and so in all of the row)
    const float k0 = (gl - g - gh * H) * ih + (lse - lse), k1 = -gh * ih, kt = g * ih;
    auto gradient = [&](float* v, int64_t c) {
#pragma unroll
      for (int e = 0; e < G; ++e) {
        // (a masked token: p = 0, and log p kept finite)
        const float low = sizeof(T) == 4 ? fmaf(fmaxf(v[e], z_low), il, -lse) : -lse;
        // (the rounding of a large lse must not carry p past 1; NaN stays)
        const float x = fmaf(v[e], ih, low);
        const float lp = x > 0.0f ? 0.0f : x;
        const float p = exp2_normal(lp * kLog2e);
        v[e] = p * fmaf(k1, fmaxf(lp, kLowLn), k0);
      }
      if (target >= c && target < c + kWaveCols) {
#pragma unroll
        for (int e = 0; e < G; ++e)
          if (GT::column(c, e) == target) v[e] += kt;
      }
      if (out) {
#pragma unroll
        for (int e = 0; e < G; ++e) v[e] = 0.0f;
      }
    };
    if (c0 + (kGradGroups - 1) * kStepCols + kWaveCols <= V) {
      typename GT::Raw raw[kGradGroups];
#pragma unroll
      for (int i = 0; i < kGradGroups; ++i)
        if (!out) raw[i] = GT::load(z + c0 + i * kStepCols);
#pragma unroll
      for (int i = 0; i < kGradGroups; ++i) {
        const int64_t c = c0 + i * kStepCols;
        float v[G];
        GT::values(raw[i], v);
        gradient(v, c);
        GT::store(dz + c, v);
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < kGradGroups; ++i) {
        const int64_t c = c0 + i * kStepCols;
        if (c >= V) break;
        float v[G];
        if (c + kWaveCols <= V) {
          GT::values(GT::load(z + c), v);
          gradient(v, c);
          GT::store(dz + c, v);
        } else {
          load_tail(z, c, V, v);
          gradient(v, c);
          store_tail(dz, c, V, v);
        }
      }
    }
  }
}

// Work-groups a chip full of streaming work wants, and the most a launch takes
// (tasks beyond it are walked by the same work-groups).  Calls without alternatives
// in us at 256, 512, 1024, 2048:
//   300 x 32003 bf16   14   17  16  18     300 x 152064 bf16  37  32  29  31
//   501 x 32003 fp32   15   19  20  21     501 x 152064 fp32  49  53  54  56
//   600 x 32003 fp32   18   18  22  24    1000 x 152064 bf16  58  58  64  66
// 512 is the middle: 256 is up to a fifth faster where a row has few pieces, and up
// to a fifth slower on few long rows.
constexpr int64_t kFill = 512;
constexpr int64_t kMaxGrid = 1 << 20;

template <class T>
hipError_t launch_rows(const LogprobArgs& a, const LogprobPlan& p, char* ws, hipStream_t s) {
  float* states = reinterpret_cast<float*>(ws);
  u64* keys = reinterpret_cast<u64*>(ws + p.off_keys);
  const int64_t tasks = a.n_tok * p.n_split;
  const dim3 grid((unsigned)(tasks < kMaxGrid ? tasks : kMaxGrid));
  const dim3 jgrid((unsigned)(a.n_tok < kMaxGrid ? a.n_tok : kMaxGrid));
  if (a.n_top > 0) {
    hipLaunchKernelGGL((logprob_rows_kernel<T, true>), grid, dim3(kThreads), 0, s, a, p.n_split,
                       p.piece, states, keys);
    if (p.n_split > 1)
      hipLaunchKernelGGL((logprob_join_kernel<T, true>), jgrid, dim3(64), 0, s, a, p.n_split,
                         states, keys);
  } else {
    hipLaunchKernelGGL((logprob_rows_kernel<T, false>), grid, dim3(kThreads), 0, s, a, p.n_split,
                       p.piece, states, keys);
    if (p.n_split > 1)
      hipLaunchKernelGGL((logprob_join_kernel<T, false>), jgrid, dim3(64), 0, s, a, p.n_split,
                         states, keys);
  }
  return hipGetLastError();
}

template <class T>
hipError_t launch_grad(const LogprobGradArgs& a, hipStream_t s) {
  const int n_pieces = (int)((a.vocab + grad_cols(sizeof(T)) - 1) / grad_cols(sizeof(T)));
  const int64_t tasks = a.n_tok * n_pieces;
  hipLaunchKernelGGL((logprob_grad_kernel<T>), dim3((unsigned)(tasks < kMaxGrid ? tasks : kMaxGrid)),
                     dim3(kThreads), 0, s, a, n_pieces);
  return hipGetLastError();
}

}  // namespace

LogprobPlan make_logprob_plan(int64_t n_tok, int64_t vocab, int n_top) {
  LogprobPlan p{};
  // whole steps of a work-group per piece, and no more pieces than fill the chip
  const int64_t steps = (vocab + kStepCols - 1) / kStepCols;
  int64_t want = n_tok > 0 ? (kFill + n_tok - 1) / n_tok : 1;
  if (want > steps) want = steps;
  if (want < 1) want = 1;
  const int64_t per = (steps + want - 1) / want;
  p.piece = per * kStepCols;
  p.n_split = (int)((steps + per - 1) / per);
  if (p.n_split > 1) {
    p.off_keys = (size_t)round_up(n_tok * p.n_split * 12, 256);
    p.total = p.off_keys + (size_t)round_up(n_tok * p.n_split * n_top * 8, 256);
  }
  return p;
}

hipError_t launch_token_logprob(const LogprobArgs& a, bool f32, const LogprobPlan& p, char* ws,
                                hipStream_t s) {
  return f32 ? launch_rows<float>(a, p, ws, s) : launch_rows<uint16_t>(a, p, ws, s);
}

hipError_t launch_token_logprob_backward(const LogprobGradArgs& a, bool f32, hipStream_t s) {
  return f32 ? launch_grad<float>(a, s) : launch_grad<uint16_t>(a, s);
}

}  // namespace logra
