// logra_sample_tokens: one token per row of logits, from a given random number,
// with temperature, top-k, top-p and min-p, on gfx950.
//
// Mathematics.  Every cut is a prefix of the tokens in descending order of their
// logits, and so is the draw: the first token whose cumulative mass exceeds u M.
// So a row needs no sort, only "where does the cumulative count (or mass) of this
// order reach a target", up to four times.  With X = (max - z) 64 log2(e) / tau the
// weight of a token is 2^(-X / 64), and bin b = floor(X) holds the weights in
// (2^(-(b + 1) / 64), 2^(-b / 64)]: 4096 bins, 64 octaves of them, hold all that can
// matter (what lies below 2^-64 of the largest weight only counts).  A bin keeps its
// tokens' number and the integer sum of 2^(-frac(X) / 64) in units of 2^-45 (fewer
// bits for vocabularies past 2^18), so the sums are exact and do not depend on the
// order of the atomics, while every token keeps a relative precision of 2^-46
// whatever its octave.  X and the exponential (a polynomial of degree 5 on [0, 1/64)
// of an octave, 2e-15) are fp64: a draw then hits a border of the cumulative masses
// wrongly about once in 10^10, where fp32 masses would in one row of a hundred.
// Scanning the bins gives the bin of a target; inside it the keys (the order-
// preserving bits of the logits) are binned again, up to twice more, until a bin
// holds one logit, whose tokens then go by their index.
#include <math.h>

#include "common.hpp"
#include "internal.hpp"
#include "step/internal_step.hpp"

namespace logra {

namespace {

typedef unsigned long long u64;

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kBins = 4096;
constexpr int kPer = kBins / kThreads;     // bins of a thread in a scan
constexpr double kFar = (double)kBins;     // X of tokens that only count

template <bool F32>
struct Row {
  static constexpr int kE = F32 ? 4 : 8;   // elements of 16 bytes
  const u32x4* p;
  int V, n_vec;
};

// The E logits of vector v of a row; those past its end read as masked tokens.
template <bool F32>
__device__ __forceinline__ void logits_of(const u32x4& q, int v, int V, float* z) {
  constexpr int E = Row<F32>::kE;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    z[e] = F32 ? __uint_as_float(q[e & 3]) : (e & 1) ? bf16_hi(q[e >> 1]) : bf16_lo(q[e >> 1]);
  }
  if (__builtin_expect((v + 1) * E > V, 0)) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (v * E + e >= V) z[e] = -INFINITY;
  }
}

// f(z, index) for every logit of the row.
template <bool F32, class F>
__device__ __forceinline__ void for_each(const Row<F32>& r, F f) {
  constexpr int E = Row<F32>::kE;
  constexpr int U = 4;
  for (int v0 = (int)threadIdx.x; v0 < r.n_vec; v0 += U * kThreads) {
    u32x4 q[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int v = v0 + i * kThreads;
      q[i] = r.p[v < r.n_vec ? v : v0];
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int v = v0 + i * kThreads;
      if (v < r.n_vec) {
        float z[E];
        logits_of<F32>(q[i], v, r.V, z);
#pragma unroll
        for (int e = 0; e < E; ++e) f(z[e], v * E + e);
      }
    }
  }
}

// A float's bits in its order (zeros of both signs are one value).
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t b = __float_as_uint(z + 0.0f);
  return b ^ ((b & 0x80000000u) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key ^ ((key & 0x80000000u) ? 0x80000000u : 0xFFFFFFFFu));
}

// What a row's weights are formed with.
struct Scale {
  double m, l64;      // largest logit, 64 log2(e) / tau
  double unit;        // 2^bits, bits of a weight's integer
};
__device__ __forceinline__ double x_of(float z, const Scale& c) { return (c.m - (double)z) * c.l64; }

// round(2^(-r / 64) unit) for r in [0, 1): the series of e^t, t = -r ln(2) / 64.
__device__ __forceinline__ u64 weight_of(double r, const Scale& c) {
  constexpr double t = -0.010830424696249145;      // -ln(2) / 64
  constexpr double c1 = t, c2 = c1 * t / 2, c3 = c2 * t / 3, c4 = c3 * t / 4, c5 = c4 * t / 5;
  double p = fma(c5, r, c4);
  p = fma(p, r, c3);
  p = fma(p, r, c2);
  p = fma(p, r, c1);
  p = fma(p, r, 1.0);
  // adding 2^52 leaves the rounded integer in the low bits of the mantissa
  const double q = fma(p, c.unit, 0x1p52);
  return (u64)__double_as_longlong(q) & 0xFFFFFFFFFFFFFull;
}
// What an integer of bin b stands for.
__device__ __forceinline__ double step_of(int b, const Scale& c) {
  return exp2(-(double)b / 64.0) / c.unit;
}

// LDS of a row.  cum and num hold the bins' cumulative masses and numbers once
// scanned; mass and cnt are the bins while they fill (again for each refinement).
struct Lds {
  u64 mass[kBins];
  uint32_t cnt[kBins];
  double cum[kBins];
  uint32_t num[kBins];
  double wave_d[kWaves];
  u64 wave_q[kWaves];
  uint32_t wave_u[kWaves], wave_v[kWaves];
  uint32_t found;
  double at_d;
  uint32_t at_u;
  u64 at_q;
};

// ------------------------------------------------------------------ over the work-group
template <class T, class F>
__device__ __forceinline__ T reduce(T x, T* lds, F f) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x = f(x, __shfl_xor(x, off));
  if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = x;
  __syncthreads();
  x = lds[0];
  for (int i = 1; i < kWaves; ++i) x = f(x, lds[i]);
  __syncthreads();
  return x;
}
// Sum over the threads before this one (a fixed order).
template <class T>
__device__ __forceinline__ T before_me(T x, T* lds) {
  T incl = x;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const T o = __shfl_up(incl, off);
    if ((int)(threadIdx.x % 64) >= off) incl += o;
  }
  if (threadIdx.x % 64 == 63) lds[threadIdx.x / 64] = incl;
  __syncthreads();
  T base = 0;
  for (int i = 0; i < (int)(threadIdx.x / 64); ++i) base += lds[i];
  __syncthreads();
  const T up = __shfl_up(incl, 1);
  return base + (threadIdx.x % 64 ? up : T(0));
}

// A target: a count to reach, or a mass to reach (or exceed).
enum Mode { kCount, kReach, kExceed };
struct Target {
  Mode mode;
  uint32_t count;
  double mass;
  __device__ __forceinline__ bool met(double c, uint32_t n) const {
    return mode == kCount ? n >= count : mode == kReach ? c >= mass : c > mass;
  }
};
// Where the order meets a target: the cumulative mass and number there, and the token.
struct Place {
  double mass;
  uint32_t rank;
  uint32_t key;
  int index;
};

// First of n entries that meets the target; -1 where none does.  at(b) gives the pair
// (mass, number) up to and including entry b.
template <class F>
__device__ __forceinline__ int first_met(Lds& s, const Target& t, F at) {
  if (threadIdx.x == 0) s.found = 0xFFFFFFFFu;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = (int)threadIdx.x * kPer + i;
    double c;
    uint32_t n;
    at(b, &c, &n);
    if (t.met(c, n)) {
      atomicMin(&s.found, (uint32_t)b);
      break;
    }
  }
  __syncthreads();
  const uint32_t f = s.found;
  __syncthreads();
  return f == 0xFFFFFFFFu ? -1 : (int)f;
}

// The j-th token (j >= 1, by index) with logit key `key`.
template <bool F32>
__device__ int nth_equal(const Row<F32>& r, Lds& s, uint32_t key, uint32_t j) {
  constexpr int E = Row<F32>::kE;
  uint32_t done = 0;
  if (threadIdx.x == 0) s.found = 0;
  for (int v0 = 0; v0 < r.n_vec; v0 += kThreads) {
    const int v = v0 + (int)threadIdx.x;
    uint32_t mine = 0, bits = 0;
    if (v < r.n_vec) {
      float z[E];
      logits_of<F32>(r.p[v], v, r.V, z);
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (z[e] > -INFINITY && key_of(z[e]) == key) {
          ++mine;
          bits |= 1u << e;
        }
    }
    const uint32_t before = done + before_me(mine, s.wave_u);
    if (before < j && before + mine >= j) {
      uint32_t left = j - before;
      int e = 0;
      for (;; ++e)
        if ((bits >> e & 1) && --left == 0) break;
      s.found = (uint32_t)(v * E + e);
    }
    done += reduce(mine, s.wave_u, [](uint32_t a, uint32_t b) { return a + b; });
    if (done >= j) break;       // (the same in every thread)
  }
  __syncthreads();
  const int f = (int)s.found;
  __syncthreads();
  return f;
}

// The place inside bin b where the order meets a target that the bin meets: the bin's
// keys are binned again until one key is left.
template <bool F32>
__device__ Place refine(const Row<F32>& r, Lds& s, const Scale& c, int b, const Target& t,
                        bool want_index) {
  const double before = b ? s.cum[b - 1] : 0.0, step = step_of(b, c);
  const uint32_t n_before = b ? s.num[b - 1] : 0u;
  uint32_t lo = 0xFFFFFFFFu, hi = 0;
  for_each<F32>(r, [&](float z, int) {
    const double X = x_of(z, c);
    if (X < kFar && (int)X == b) {
      const uint32_t k = key_of(z);
      lo = k < lo ? k : lo;
      hi = k > hi ? k : hi;
    }
  });
  lo = reduce(lo, s.wave_u, [](uint32_t x, uint32_t y) { return x < y ? x : y; });
  hi = reduce(hi, s.wave_u, [](uint32_t x, uint32_t y) { return x > y ? x : y; });
  u64 q_done = 0;
  uint32_t n_done = 0;
  for (;;) {
    const uint32_t range = hi - lo;
    const int shift = range < (uint32_t)kBins ? 0 : 32 - __clz((int)range) - 12;
    for (int i = (int)threadIdx.x; i < kBins; i += kThreads) {
      s.mass[i] = 0;
      s.cnt[i] = 0;
    }
    __syncthreads();
    for_each<F32>(r, [&](float z, int) {
      const double X = x_of(z, c);
      const uint32_t k = key_of(z);
      if (X < kFar && (int)X == b && k >= lo && k <= hi) {
        const uint32_t sub = (hi - k) >> shift;
        atomicAdd(&s.mass[sub], weight_of(X - (double)b, c));
        atomicAdd(&s.cnt[sub], 1u);
      }
    });
    __syncthreads();
    // cumulative sums of the sub-bins, each in its own place
    u64 q[kPer], qs = 0;
    uint32_t n[kPer], ns = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      q[i] = qs += s.mass[threadIdx.x * kPer + i];
      n[i] = ns += s.cnt[threadIdx.x * kPer + i];
    }
    const u64 q0 = q_done + before_me(qs, s.wave_q);
    const uint32_t n0 = n_done + before_me(ns, s.wave_u);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      s.mass[threadIdx.x * kPer + i] = q0 + q[i];
      s.cnt[threadIdx.x * kPer + i] = n0 + n[i];
    }
    __syncthreads();
    auto subs = [&](int i, double* m, uint32_t* k) {
      *m = before + step * (double)s.mass[i];
      *k = n_before + s.cnt[i];
    };
    int sub = first_met(s, t, subs);
    if (sub < 0)    // (a mass that a rounding of the last sum leaves unmet: the last key)
      sub = first_met(s, Target{kCount, n_before + s.cnt[kBins - 1], 0.0}, subs);
    const u64 q_to = s.mass[sub];
    const uint32_t n_to = s.cnt[sub];
    const u64 q_from = sub ? s.mass[sub - 1] : q_done;
    const uint32_t n_from = sub ? s.cnt[sub - 1] : n_done;
    __syncthreads();
    if (shift == 0) {
      const uint32_t key = hi - (uint32_t)sub;
      const u64 w = (q_to - q_from) / (n_to - n_from);       // the same for each
      uint32_t a = 1, z = n_to - n_from;                     // the first j that meets it
      while (a < z) {
        const uint32_t mid = a + (z - a) / 2;
        if (t.met(before + step * (double)(q_from + w * mid), n_before + n_from + mid))
          z = mid;
        else
          a = mid + 1;
      }
      Place p;
      p.mass = before + step * (double)(q_from + w * a);
      p.rank = n_before + n_from + a;
      p.key = key;
      p.index = want_index ? nth_equal<F32>(r, s, key, a) : -1;
      return p;
    }
    q_done = q_from;
    n_done = n_from;
    hi -= (uint32_t)sub << shift;
    const uint32_t low = hi - ((1u << shift) - 1);
    lo = low > lo && low <= hi ? low : lo;
  }
}

// ------------------------------------------------------------------ a row
template <bool F32>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs a, double unit) {
  __shared__ Lds s;
  const int64_t t = (int64_t)blockIdx.x;
  auto put = [&](int64_t token, float logp, float logq, uint32_t kept) {
    if (threadIdx.x != 0) return;
    a.token[t] = token;
    if (a.logp != nullptr) a.logp[t] = logp;
    if (a.logq != nullptr) a.logq[t] = logq;
    if (a.kept != nullptr) a.kept[t] = (int32_t)kept;
  };
  const float u = a.u[t];
  if (!(u >= 0.0f && u < 1.0f)) return put(-1, 0.0f, 0.0f, 0);
  const float tau = a.tau_rows != nullptr ? a.tau_rows[t] : a.tau;
  const float top_p = a.top_p_rows != nullptr ? a.top_p_rows[t] : a.top_p;
  const float min_p = a.min_p_rows != nullptr ? a.min_p_rows[t] : a.min_p;
  const int32_t top_k = a.top_k_rows != nullptr ? a.top_k_rows[t] : a.top_k;
  if (!(tau > 0.0f && tau < INFINITY && top_p > 0.0f && top_p <= 1.0f && min_p >= 0.0f &&
        min_p <= 1.0f))
    return put(-1, NAN, NAN, 0);
  Row<F32> r;
  r.V = a.vocab;
  r.n_vec = (a.vocab + Row<F32>::kE - 1) / Row<F32>::kE;
  r.p = reinterpret_cast<const u32x4*>(static_cast<const char*>(a.z) +
                                       t * a.ld * (F32 ? 4 : 2));
  // the largest logit; a NaN shows in `bad`
  float m = -INFINITY;
  uint32_t bad = 0;
  for_each<F32>(r, [&](float z, int) {
    m = fmaxf(m, z);
    bad |= z != z;
  });
  m = reduce(m, reinterpret_cast<float*>(s.wave_u), [](float x, float y) { return fmaxf(x, y); });
  bad = reduce(bad, s.wave_u, [](uint32_t x, uint32_t y) { return x | y; });
  if (bad || !(fabsf(m) < INFINITY)) return put(-1, NAN, NAN, 0);
  Scale c;
  c.m = (double)m;
  c.l64 = 64.0 * 1.4426950408889634074 / (double)tau;
  c.unit = unit;
  // bins, and what only counts
  for (int i = (int)threadIdx.x; i < kBins; i += kThreads) {
    s.mass[i] = 0;
    s.cnt[i] = 0;
  }
  __syncthreads();
  const double x_min = min_p > 0.0f ? -64.0 * log2((double)min_p) : INFINITY;
  uint32_t n_far = 0, n_min = 0;
  for_each<F32>(r, [&](float z, int) {
    if (z > -INFINITY) {
      const double X = x_of(z, c);
      n_min += X <= x_min;
      if (X < kFar) {
        const int b = (int)X;
        atomicAdd(&s.mass[b], weight_of(X - (double)b, c));
        atomicAdd(&s.cnt[b], 1u);
      } else {
        ++n_far;
      }
    }
  });
  auto sum = [](uint32_t x, uint32_t y) { return x + y; };
  n_far = reduce(n_far, s.wave_u, sum);
  n_min = reduce(n_min, s.wave_u, sum);
  // cumulative masses and numbers
  {
    double d[kPer], ds = 0;
    uint32_t n[kPer], ns = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = (int)threadIdx.x * kPer + i;
      d[i] = ds += (double)s.mass[b] * step_of(b, c);
      n[i] = ns += s.cnt[b];
    }
    const double d0 = before_me(ds, s.wave_d);
    const uint32_t n0 = before_me(ns, s.wave_u);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      s.cum[threadIdx.x * kPer + i] = d0 + d[i];
      s.num[threadIdx.x * kPer + i] = n0 + n[i];
    }
  }
  __syncthreads();
  const double total = s.cum[kBins - 1];
  const uint32_t near = s.num[kBins - 1], live = near + n_far;
  auto bins = [&](int b, double* x, uint32_t* n) {
    *x = s.cum[b];
    *n = s.num[b];
  };
  auto find = [&](const Target& tg, bool want_index) {
    int b = first_met(s, tg, bins);
    if (b < 0)      // (unmet by a rounding: the last token that has a weight)
      b = first_met(s, Target{kCount, near, 0.0}, bins);
    return refine<F32>(r, s, c, b, tg, want_index);
  };
  auto mass_of = [&](uint32_t k) {
    return k >= near ? total : find(Target{kCount, k, 0.0}, false).mass;
  };
  const uint32_t k1 = top_k > 0 && (uint32_t)top_k < live ? (uint32_t)top_k : live;
  const double m1 = mass_of(k1);
  uint32_t kept = k1;
  double M = m1;
  if (top_p < 1.0f) {
    const Place p = find(Target{kReach, 0, (double)top_p * m1}, false);
    if (p.rank < kept) {
      kept = p.rank;
      M = p.mass;
    }
  }
  if (n_min < kept) {       // (at least the largest logit passes min_p)
    kept = n_min;
    M = mass_of(kept);
  }
  const Place p = find(Target{kExceed, 0, (double)u * M}, true);
  const double lw = -x_of(value_of(p.key), c) * (0.69314718055994530942 / 64.0);
  put(p.index, (float)(lw - log(total)), (float)(lw - log(M)), kept);
}

}  // namespace

size_t sample_ws_bytes(int64_t, int64_t) { return 0; }

hipError_t launch_sample(const SampleArgs& a, bool f32, char*, hipStream_t s) {
  // a bin's sum of `vocab` integers up to 2^bits stays below 2^63
  int bits = 45;
  while (bits > 32 && ((double)a.vocab * exp2((double)bits)) > 0x1p63) --bits;
  const double unit = exp2((double)bits);
  auto kernel = f32 ? sample_kernel<true> : sample_kernel<false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)a.n_tok), dim3(kThreads), 0, s, a, unit);
  return hipGetLastError();
}

}  // namespace logra
