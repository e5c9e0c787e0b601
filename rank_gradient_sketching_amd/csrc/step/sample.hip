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
// of an octave, 2e-15) are fp64, which costs a fused step what fp32 does: a draw then
// hits a border of the cumulative masses wrongly about once in 10^10, where fp32
// masses would in one row of a hundred.
// Scanning the bins gives, for each target, the bin (or, where a target depends on
// one that is not resolved yet, the few bins) that it lies in.  Their tokens, usually
// some tens, are gathered from the row, sorted by logit and index, and resolve all
// targets at once.  A row whose bins hold more than fit there (logits nearly equal, or
// many ties) takes them one by one: the keys (the order-preserving bits of the logits)
// of a bin are binned again, up to three times, until one logit is left, whose tokens
// then go by their index.
//
// Bound.  A row is read twice or three times (maximum, bins, gathered list), the later
// times out of the caches, and what each logit costs in between (an fp64 product, the
// polynomial, two LDS atomics: some 40 issue slots a wave and logit) is far more than
// its two bytes.  512 x 152064 bf16 takes 147 us: 25 the maximum, 40 the bins, 7 their
// scan, 25 the gathering and up to 15 the resolving; the other 35 are not attributed.  Read
// once at 7.2 TB/s it would take 22.  A work-group of 512 threads holds 49 KB of bins, so two
// share a CU and one's barriers hide behind the other's logits; four of 256 threads do
// not fit, one of 1024 took 184 us.  Few rows leave CUs idle, so they are cut into
// pieces: 8 x 152064 takes 39 us (6 + 9 + 25: maximum, bins, pick) against 57 with a
// work-group per row; the pick's own gathering (9 us) and its loading and scanning of
// the bins (8) are latency.
#include <math.h>

#include "common.hpp"
#include "internal.hpp"
#include "step/internal_step.hpp"

namespace logra {

namespace {

typedef unsigned long long u64;

constexpr int kBins = 4096;
constexpr int kSpare = 64;                 // bins for what lies past them, one per lane
constexpr double kFar = (double)kBins;     // X of tokens that only count
constexpr int kList = 2048;                // tokens that are gathered and sorted
constexpr int kSubs = 1024;                // bins of a refinement
constexpr int kMaxWaves = 16;

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
  for (int e = 0; e < E; ++e)
    z[e] = F32 ? __uint_as_float(q[e & 3]) : (e & 1) ? bf16_hi(q[e >> 1]) : bf16_lo(q[e >> 1]);
  if (__builtin_expect((uint32_t)(v + 1) * E > (uint32_t)V, 0)) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if ((uint32_t)v * E + e >= (uint32_t)V) z[e] = -INFINITY;
  }
}

// f(z) for the logits of vectors [v0, v1) of the row, U loads in flight.
template <int THREADS, int U, bool F32, class F>
__device__ __forceinline__ void for_each(const Row<F32>& r, int v0, int v1, F f) {
  constexpr int E = Row<F32>::kE;
  for (int at = v0 + (int)threadIdx.x; at < v1; at += U * THREADS) {
    u32x4 q[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int v = at + i * THREADS;
      q[i] = r.p[v < v1 ? v : at];
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int v = at + i * THREADS;
      if (v < v1) {
        float z[E];
        logits_of<F32>(q[i], v, r.V, z);
#pragma unroll
        for (int e = 0; e < E; ++e) f(z[e]);
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

// What a row's weights are formed with.  w: the polynomial's coefficients times 2^bits,
// bits of a weight's integer, and on the last one 2^52, which leaves the rounded integer
// in the low bits of the mantissa.
struct Scale {
  double m, l64;      // largest logit, 64 log2(e) / tau
  double w[6];
  double unit;        // 2^bits
};
__device__ __forceinline__ Scale scale_of(float m, float tau, double unit) {
  constexpr double t = -0.010830424696249145;      // -ln(2) / 64
  constexpr double c1 = t, c2 = c1 * t / 2, c3 = c2 * t / 3, c4 = c3 * t / 4, c5 = c4 * t / 5;
  Scale s;
  s.l64 = 64.0 * 1.4426950408889634074 / (double)tau;
  s.m = (double)m;
  s.w[0] = unit + 0x1p52;
  s.w[1] = c1 * unit;
  s.w[2] = c2 * unit;
  s.w[3] = c3 * unit;
  s.w[4] = c4 * unit;
  s.w[5] = c5 * unit;
  s.unit = unit;
  return s;
}
__device__ __forceinline__ double x_of(float z, const Scale& s) {
  return (s.m - (double)z) * s.l64;
}

// round(2^(-frac(X) / 64) unit) + kBias, the pattern of 2^52: sums of these wrap round
// 2^64, and n kBias taken off a sum of n leaves the sum of the integers.
constexpr u64 kBias = 0x4330000000000000ull;
__device__ __forceinline__ u64 weight_of(double X, const Scale& c) {
  const double r = __builtin_amdgcn_fract(X);
  double p = fma(c.w[5], r, c.w[4]);
  p = fma(p, r, c.w[3]);
  p = fma(p, r, c.w[2]);
  p = fma(p, r, c.w[1]);
  p = fma(p, r, c.w[0]);
  return (u64)__double_as_longlong(p);
}
// What an integer of bin b stands for.
__device__ __forceinline__ double step_of(int b, const Scale& c) {
  return exp2(-(double)b / 64.0) / c.unit;
}

// LDS of a row, 65 KB, so that two rows share a CU and one's loads cover the other's
// arithmetic.
struct Lds {
  union {
    u64 mass[kBins + kSpare];   // while the bins fill
    double cum[kBins];       // then: cumulative masses
  };
  uint32_t num[kBins + kSpare];  // numbers of tokens, then cumulative
  double group_cum[64];      // of every 64th bin
  uint32_t group_num[64];
  union {
    u64 list[kList];         // ~key, index
    struct {
      u64 mass[kSubs];
      uint32_t num[kSubs];
    } sub;
  };
  union {
    double wave_d[kMaxWaves];
    u64 wave_q[kMaxWaves];
  };
  uint32_t wave_u[kMaxWaves];
  double at_mass;
  uint32_t at_rank, at_key, n_list;
  int at_index;
};

// ------------------------------------------------------------------ over the work-group
template <int THREADS, class T, class F>
__device__ __forceinline__ T reduce(T x, T* lds, F f) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x = f(x, __shfl_xor(x, off));
  if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = x;
  __syncthreads();
  x = lds[0];
#pragma unroll
  for (int i = 1; i < THREADS / 64; ++i) x = f(x, lds[i]);
  __syncthreads();
  return x;
}
struct Add {
  template <class T>
  __device__ T operator()(T a, T b) const { return a + b; }
};
// Sum over the threads before this one (a fixed order).
template <int THREADS, class T>
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
#pragma unroll
  for (int i = 0; i < THREADS / 64; ++i)
    if (i < (int)(threadIdx.x / 64)) base += lds[i];
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

// First of N entries that meets the target; -1 where none does.  at(b) gives the pair
// (mass, number) up to and including entry b.
template <int THREADS, int N, class F>
__device__ __forceinline__ int first_met(Lds& s, const Target& t, F at) {
  constexpr int kPer = N / THREADS;
  uint32_t f = 0xFFFFFFFFu;
#pragma unroll
  for (int i = kPer - 1; i >= 0; --i) {
    const int b = (int)threadIdx.x * kPer + i;
    double c;
    uint32_t n;
    at(b, &c, &n);
    if (t.met(c, n)) f = (uint32_t)b;
  }
  return (int)reduce<THREADS>(f, s.wave_u, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}

// ------------------------------------------------------------------ one target at a time
// The j-th token (j >= 1, by index) with logit key `key`.
template <int THREADS, bool F32>
__device__ __noinline__ int nth_equal(Row<F32> r, Lds& s, uint32_t key, uint32_t j) {
  constexpr int E = Row<F32>::kE;
  uint32_t done = 0;
  if (threadIdx.x == 0) s.at_index = 0;
  for (int v0 = 0; v0 < r.n_vec; v0 += THREADS) {
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
    const uint32_t before = done + before_me<THREADS>(mine, s.wave_u);
    if (before < j && before + mine >= j) {
      uint32_t left = j - before;
      int e = 0;
      for (;; ++e)
        if ((bits >> e & 1) && --left == 0) break;
      s.at_index = v * E + e;
    }
    done += reduce<THREADS>(mine, s.wave_u, Add());
    if (done >= j) break;       // (the same in every thread)
  }
  __syncthreads();
  const int f = s.at_index;
  __syncthreads();
  return f;
}

// The place inside bin b where the order meets a target that the bin meets: the bin's
// keys are binned again until one key is left.
template <int THREADS, bool F32>
__device__ __noinline__ Place refine(Row<F32> r, Lds& s, Scale c, int b, Target t,
                                     bool want_index) {
  constexpr int kPer = kSubs / THREADS;
  const double before = b ? s.cum[b - 1] : 0.0, step = step_of(b, c);
  const uint32_t n_before = b ? s.num[b - 1] : 0u;
  uint32_t lo = 0xFFFFFFFFu, hi = 0;
  for_each<THREADS, 4>(r, 0, r.n_vec, [&](float z) {
    const double X = x_of(z, c);
    if (X < kFar && (int)X == b) {
      const uint32_t k = key_of(z);
      lo = k < lo ? k : lo;
      hi = k > hi ? k : hi;
    }
  });
  lo = reduce<THREADS>(lo, s.wave_u, [](uint32_t x, uint32_t y) { return x < y ? x : y; });
  hi = reduce<THREADS>(hi, s.wave_u, [](uint32_t x, uint32_t y) { return x > y ? x : y; });
  u64 q_done = 0;
  uint32_t n_done = 0;
  for (;;) {
    const uint32_t range = hi - lo;
    const int shift = range < (uint32_t)kSubs ? 0 : 32 - __clz((int)range) - 10;
    for (int i = (int)threadIdx.x; i < kSubs; i += THREADS) {
      s.sub.mass[i] = 0;
      s.sub.num[i] = 0;
    }
    __syncthreads();
    for_each<THREADS, 4>(r, 0, r.n_vec, [&](float z) {
      const double X = x_of(z, c);
      const uint32_t k = key_of(z);
      if (X < kFar && (int)X == b && k >= lo && k <= hi) {
        const uint32_t sub = (hi - k) >> shift;
        atomicAdd(&s.sub.mass[sub], weight_of(X, c) - kBias);
        atomicAdd(&s.sub.num[sub], 1u);
      }
    });
    __syncthreads();
    // cumulative sums of the sub-bins, each in its own place
    u64 q[kPer], qs = 0;
    uint32_t n[kPer], ns = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      q[i] = qs += s.sub.mass[threadIdx.x * kPer + i];
      n[i] = ns += s.sub.num[threadIdx.x * kPer + i];
    }
    const u64 q0 = q_done + before_me<THREADS>(qs, s.wave_q);
    const uint32_t n0 = n_done + before_me<THREADS>(ns, s.wave_u);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      s.sub.mass[threadIdx.x * kPer + i] = q0 + q[i];
      s.sub.num[threadIdx.x * kPer + i] = n0 + n[i];
    }
    __syncthreads();
    auto subs = [&](int i, double* m, uint32_t* k) {
      *m = before + step * (double)s.sub.mass[i];
      *k = n_before + s.sub.num[i];
    };
    int sub = first_met<THREADS, kSubs>(s, t, subs);
    if (sub < 0)    // (a mass that a rounding of the last sum leaves unmet: the last key)
      sub = first_met<THREADS, kSubs>(s, Target{kCount, n_before + s.sub.num[kSubs - 1], 0.0},
                                      subs);
    const u64 q_to = s.sub.mass[sub];
    const uint32_t n_to = s.sub.num[sub];
    const u64 q_from = sub ? s.sub.mass[sub - 1] : q_done;
    const uint32_t n_from = sub ? s.sub.num[sub - 1] : n_done;
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
      p.index = want_index ? nth_equal<THREADS>(r, s, key, a) : -1;
      return p;
    }
    q_done = q_from;
    n_done = n_from;
    hi -= (uint32_t)sub << shift;
    const uint32_t low = hi - ((1u << shift) - 1);
    lo = low > lo && low <= hi ? low : lo;
  }
}

// What cuts a row's order, and its draw.
struct Cuts {
  double p, u, total;
  uint32_t k1, min, near;      // near: tokens in the bins
  bool k, by_p, by_min;        // which cuts there are
};
// The bin where the order meets a target: every wave finds it for itself, first the 64
// bins that hold it, then the one.
__device__ __forceinline__ int bin_of(const Lds& s, const Target& t, uint32_t near) {
  const int lane = threadIdx.x & 63;
  u64 met = __ballot(t.met(s.group_cum[lane], s.group_num[lane]));
  // (unmet by a rounding: the last bin that holds a token)
  const Target last{kCount, near, 0.0};
  const Target& u = met ? t : last;
  if (met == 0) met = __ballot(u.met(s.group_cum[lane], s.group_num[lane]));
  const int g = (__ffsll(met) - 1) * 64;
  return g + __ffsll(__ballot(u.met(s.cum[g + lane], s.num[g + lane]))) - 1;
}
template <int THREADS, bool F32>
__device__ __noinline__ Place one_by_one(Row<F32> r, Lds& s, Scale c, Cuts x, uint32_t* kept,
                                         double* M) {
  uint32_t k = x.k1;
  double m = x.total;
  // the cuts, then the draw: one loop, so that there is one copy of the search
  Place at{};
  for (int i = 0; i < 4; ++i) {
    Target t{kCount, k, 0.0};
    if (i == 0 && !x.k) continue;
    if (i == 1) {
      if (!x.by_p) continue;
      t = Target{kReach, 0, x.p * m};
    }
    if (i == 2) {
      if (!x.by_min || x.min >= k) continue;
      t.count = x.min;
    }
    if (i == 3) t = Target{kExceed, 0, x.u * m};
    at = refine<THREADS>(r, s, c, bin_of(s, t, x.near), t, i == 3);
    if (i == 0 || (i < 3 && at.rank < k)) {
      k = at.rank;
      m = at.mass;
    }
  }
  *kept = k;
  *M = m;
  return at;
}

// ------------------------------------------------------------------ a row
struct Settings {
  float u, tau, top_p, min_p;
  int32_t top_k;
  bool left_out, legal;
};
__device__ __forceinline__ Settings settings_of(const SampleArgs& a, int64_t t) {
  Settings g;
  g.u = a.u[t];
  g.left_out = !(g.u >= 0.0f && g.u < 1.0f);
  g.tau = a.tau_rows != nullptr ? a.tau_rows[t] : a.tau;
  g.top_p = a.top_p_rows != nullptr ? a.top_p_rows[t] : a.top_p;
  g.min_p = a.min_p_rows != nullptr ? a.min_p_rows[t] : a.min_p;
  g.top_k = a.top_k_rows != nullptr ? a.top_k_rows[t] : a.top_k;
  g.legal = g.tau > 0.0f && g.tau < INFINITY && g.top_p > 0.0f && g.top_p <= 1.0f &&
            g.min_p >= 0.0f && g.min_p <= 1.0f;
  return g;
}
struct Drawn {
  int token;
  float logp, logq;
  uint32_t kept;
};
__device__ __forceinline__ void put(const SampleArgs& a, int64_t t, const Drawn& d) {
  if (threadIdx.x != 0) return;
  a.token[t] = d.token;
  if (a.logp != nullptr) a.logp[t] = d.logp;
  if (a.logq != nullptr) a.logq[t] = d.logq;
  if (a.kept != nullptr) a.kept[t] = (int32_t)d.kept;
}
__device__ __forceinline__ Drawn left_out() { return Drawn{-1, 0.0f, 0.0f, 0}; }
__device__ __forceinline__ Drawn no_token() { return Drawn{-1, NAN, NAN, 0}; }
template <bool F32>
__device__ __forceinline__ Row<F32> row_of(const SampleArgs& a, int64_t t) {
  Row<F32> r;
  r.V = a.vocab;
  r.n_vec = (int)(((int64_t)a.vocab + Row<F32>::kE - 1) / Row<F32>::kE);
  r.p = reinterpret_cast<const u32x4*>(static_cast<const char*>(a.z) + t * a.ld * (F32 ? 4 : 2));
  return r;
}

// The largest of a thread's logits (NaN where one of them is NaN), and how many of them
// are masked.
struct Top {
  float m;
  uint32_t masked;
};
template <int THREADS, bool F32>
__device__ __forceinline__ Top top_part(const Row<F32>& r, int v0, int v1) {
  constexpr int E = Row<F32>::kE, U = 8;
  Top t{-INFINITY, 0};
  bool bad = false;
  for (int at = v0 + (int)threadIdx.x; at < v1; at += U * THREADS) {
    u32x4 q[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int v = at + i * THREADS;
      q[i] = r.p[v < v1 ? v : at];
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int v = at + i * THREADS;
      float z[E];
      logits_of<F32>(q[i], v < v1 ? v : at, r.V, z);
      float lo = z[0];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        t.m = fmaxf(t.m, z[e]);
        lo = fminf(lo, z[e]);
        bad = bad || z[e] != z[e];
      }
      if (lo == -INFINITY && v < v1) {
#pragma unroll
        for (int e = 0; e < E; ++e)      // (not those past the row's end)
          t.masked += z[e] == -INFINITY && (uint32_t)v * E + e < (uint32_t)r.V;
      }
    }
  }
  if (bad) t.m = NAN;
  return t;
}
__device__ __forceinline__ float max_or_nan(float a, float b) {
  return a != a ? a : b != b ? b : fmaxf(a, b);
}

// Tokens that are not masked, and those that pass min_p (without it: kAll).
constexpr uint32_t kAll = 0xFFFFFFFFu;
struct Counts {
  uint32_t live, min;
};
// Fills the bins with the logits of vectors [v0, v1); the number of a thread's own that
// pass min_p.  Without branches (tokens past the bins go to a spare one of the lane), so
// that the arithmetic of a vector's logits overlaps.
template <int THREADS, bool MIN, bool F32>
__device__ __forceinline__ uint32_t bin_part(const Row<F32>& r, int v0, int v1, Lds& s,
                                             const Scale& c, double x_min) {
  constexpr int E = Row<F32>::kE, U = 4;
  const int spare = kBins + (int)(threadIdx.x & 63);
  uint32_t n_min = 0;
  for (int at = v0 + (int)threadIdx.x; at < v1; at += U * THREADS) {
    u32x4 q[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int v = at + i * THREADS;
      q[i] = r.p[v < v1 ? v : at];
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int v = at + i * THREADS;
      if (v >= v1) break;
      float z[E];
      logits_of<F32>(q[i], v, r.V, z);
      double X[E];
      u64 w[E];
      int b[E];
#pragma unroll
      for (int e = 0; e < E; ++e) X[e] = x_of(z[e], c);
#pragma unroll
      for (int e = 0; e < E; ++e) b[e] = X[e] < kFar ? (int)X[e] : spare;
#pragma unroll
      for (int e = 0; e < E; ++e) w[e] = weight_of(X[e], c);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if constexpr (MIN) n_min += X[e] <= x_min;
        atomicAdd(&s.mass[b[e]], w[e]);
        atomicAdd(&s.num[b[e]], 1u);
      }
    }
  }
  return n_min;
}
// (the sum over the work-group)
template <int THREADS, bool F32>
__device__ __forceinline__ uint32_t fill_bins(const Row<F32>& r, int v0, int v1, Lds& s,
                                              const Scale& c, float min_p) {
  if (!(min_p > 0.0f)) {
    bin_part<THREADS, false>(r, v0, v1, s, c, 0.0);
    __syncthreads();
    return kAll;
  }
  return reduce<THREADS>(bin_part<THREADS, true>(r, v0, v1, s, c, -64.0 * log2((double)min_p)),
                         s.wave_u, Add());
}

// Bins that hold what the targets need: single ones and runs.
struct Wanted {
  int lo[4], hi[4];
  __device__ __forceinline__ bool has_x(double X) const { return X < kFar && has((int)X); }
  __device__ __forceinline__ bool has(int b) const {
    return (b >= lo[0] && b <= hi[0]) || (b >= lo[1] && b <= hi[1]) ||
           (b >= lo[2] && b <= hi[2]) || (b >= lo[3] && b <= hi[3]);
  }
};

// Sorts the first n entries of the list (the rest is filled up with the largest).
template <int THREADS>
__device__ __forceinline__ void sort_list(Lds& s, int n) {
  int size = 64;
  while (size < n) size <<= 1;
  for (int i = n + (int)threadIdx.x; i < size; i += THREADS) s.list[i] = ~0ull;
  __syncthreads();
  for (int k = 2; k <= size; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = (int)threadIdx.x; i < size / 2; i += THREADS) {
        const int a = 2 * i - (i & (j - 1)), b = a + j;
        const u64 x = s.list[a], y = s.list[b];
        if ((x > y) == ((a & k) == 0)) {
          s.list[a] = y;
          s.list[b] = x;
        }
      }
      __syncthreads();
    }
}

// What a thread knows of one token of the sorted list.
struct Entry {
  double mass;        // cumulative, as is the rank; 0 where there is no token
  uint32_t rank;
};
// The cumulative mass and number at a token of bin b that is the n-th of its bin, q the
// sum of the bin's integers up to it.
__device__ __forceinline__ Entry entry_of(const Lds& s, const Scale& c, int b, u64 q, uint32_t n) {
  const double before = b > 0 ? s.cum[b - 1] : 0.0;
  Entry e;
  e.rank = (b > 0 ? s.num[b - 1] : 0u) + n;
  // (the bin's last token has the bin's cumulative mass to the last bit)
  e.mass = e.rank == s.num[b] ? s.cum[b] : fmin(s.cum[b], before + step_of(b, c) * (double)q);
  return e;
}
// The kept number, their mass and the draw, from a function that resolves targets.
template <class F>
__device__ __forceinline__ Place resolve_all(const Cuts& x, uint32_t* kept, double* M, F resolve) {
  if (x.k) *M = resolve(Target{kCount, x.k1, 0.0}).mass;
  if (x.by_p) {
    const Place at = resolve(Target{kReach, 0, x.p * *M});
    if (at.rank < *kept) {
      *kept = at.rank;
      *M = at.mass;
    }
  }
  if (x.by_min && x.min < *kept) {
    *kept = x.min;
    *M = resolve(Target{kCount, x.min, 0.0}).mass;
  }
  return resolve(Target{kExceed, 0, x.u * *M});
}

// A list of at most 64 tokens, one per lane of the first wave.
__device__ __forceinline__ Place resolve_short(Lds& s, const Scale& c, const Cuts& x,
                                               const Wanted& want, int n_list, uint32_t* kept,
                                               double* M) {
  const int lane = threadIdx.x & 63;
  // (a neighbour of the wanted bins gets an entry past all others, as lanes without one)
  u64 mine = lane < n_list ? s.list[lane] : ~0ull;
  if (lane < n_list && !want.has_x(x_of(value_of(~(uint32_t)(mine >> 32)), c))) {
    mine = ~0ull;
    s.list[lane] = mine;
  }
  const u64 valid = __ballot(mine != ~0ull);
  const int n = __popcll(valid);
  int place = 0;
  for (int i = 0; i < n_list; ++i) place += s.list[i] < mine;
  if (mine == ~0ull) place = n + lane - __popcll(valid & ((1ull << lane) - 1));
  const uint32_t hi = (uint32_t)__builtin_amdgcn_ds_permute(place * 4, (int)(mine >> 32));
  const uint32_t index = (uint32_t)__builtin_amdgcn_ds_permute(place * 4, (int)mine);
  const uint32_t key = ~hi;
  const double X = x_of(value_of(key), c);
  const int b = lane < n ? (int)X : -1;
  u64 q = lane < n ? weight_of(X, c) - kBias : 0;
  uint32_t run = 1;
  const int b_before = __shfl_up(b, 1);       // (every lane takes part)
  bool head = lane == 0 || b != b_before;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const u64 o_q = __shfl_up(q, off);
    const uint32_t o_run = __shfl_up(run, off);
    const bool o_head = __shfl_up((int)head, off) != 0;
    if (lane >= off && !head) {
      q += o_q;
      run += o_run;
      head = o_head;
    }
  }
  Entry e{0.0, 0};
  if (lane < n) e = entry_of(s, c, b, q, run);
  return resolve_all(x, kept, M, [&](const Target& t) {
    const u64 met = __ballot(lane < n && t.met(e.mass, e.rank));
    const int f = met ? __ffsll(met) - 1 : n - 1;
    return Place{__shfl(e.mass, f), (uint32_t)__shfl((int)e.rank, f), (uint32_t)__shfl((int)key, f),
                 __shfl((int)index, f)};
  });
}

// A longer list: sorted in LDS, kList / THREADS consecutive tokens a thread.
template <int THREADS>
__device__ __forceinline__ Place resolve_long(Lds& s, const Scale& c, const Cuts& x,
                                              const Wanted& want, int n_list, uint32_t* kept,
                                              double* M) {
  constexpr int kMine = kList / THREADS;
  // (neighbours of the wanted bins are sorted to the end)
  uint32_t mine = 0;
  for (int i = (int)threadIdx.x; i < n_list; i += THREADS) {
    if (want.has_x(x_of(value_of(~(uint32_t)(s.list[i] >> 32)), c)))
      ++mine;
    else
      s.list[i] = ~0ull;
  }
  const int n = (int)reduce<THREADS>(mine, s.wave_u, Add());
  sort_list<THREADS>(s, n_list);
  // sums of a bin's integers and tokens up to each token, which start anew with every bin
  u64 q[kMine];
  uint32_t run[kMine];
  int bin[kMine];
  const int first = (int)threadIdx.x * kMine;
  auto x_at = [&](int i) { return x_of(value_of(~(uint32_t)(s.list[i] >> 32)), c); };
  u64 sum = 0;
  uint32_t ns = 0;
  bool head = false;         // whether a bin starts here
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    if (first + i < n) {
      const double X = x_at(first + i);
      bin[i] = (int)X;
      const int prev = i ? bin[i - 1] : first > 0 ? (int)x_at(first - 1) : -1;
      if (bin[i] != prev) {
        head = true;
        sum = 0;
        ns = 0;
      }
      sum += weight_of(X, c) - kBias;
      ++ns;
      q[i] = sum;
      run[i] = head ? ns : 0x80000000u | ns;     // (marked: lacks what came before)
    }
  }
  // sums of the bins that began in earlier threads: a scan that restarts at heads
  u64 in_sum = sum;
  uint32_t in_run = ns | (head ? 0x80000000u : 0u);
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const u64 o_sum = __shfl_up(in_sum, off);
    const uint32_t o_run = __shfl_up(in_run, off);
    if ((int)(threadIdx.x % 64) >= off && !(in_run & 0x80000000u)) {
      in_sum += o_sum;
      in_run += o_run;       // (takes the mark over)
    }
  }
  if (threadIdx.x % 64 == 63) {
    s.wave_q[threadIdx.x / 64] = in_sum;
    s.wave_u[threadIdx.x / 64] = in_run;
  }
  __syncthreads();
  u64 w_sum = 0;
  uint32_t w_run = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w)
    if (w < (int)(threadIdx.x / 64)) {
      const bool anew = (s.wave_u[w] & 0x80000000u) != 0;
      w_sum = (anew ? 0 : w_sum) + s.wave_q[w];
      w_run = (anew ? 0 : w_run) + (s.wave_u[w] & 0x7FFFFFFFu);
    }
  __syncthreads();
  u64 e_sum = __shfl_up(in_sum, 1);
  uint32_t e_run = __shfl_up(in_run, 1);
  if (threadIdx.x % 64 == 0) {
    e_sum = w_sum;
    e_run = w_run;
  } else if (!(e_run & 0x80000000u)) {
    e_sum += w_sum;
    e_run += w_run;
  }
  e_run &= 0x7FFFFFFFu;
  Entry e[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    e[i] = Entry{0.0, 0};
    if (first + i < n) {
      const bool lacks = (run[i] & 0x80000000u) != 0;
      e[i] = entry_of(s, c, bin[i], q[i] + (lacks ? e_sum : 0),
                      (run[i] & 0x7FFFFFFFu) + (lacks ? e_run : 0));
    }
  }
  // the first rank that meets a target, and what stands there
  return resolve_all(x, kept, M, [&](const Target& t) {
    uint32_t f = 0xFFFFFFFFu;
#pragma unroll
    for (int i = kMine - 1; i >= 0; --i)
      if (first + i < n && t.met(e[i].mass, e[i].rank)) f = e[i].rank;
    f = reduce<THREADS>(f, s.wave_u, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
#pragma unroll
    for (int i = 0; i < kMine; ++i)
      if (first + i < n && (e[i].rank == f || (f == 0xFFFFFFFFu && first + i == n - 1))) {
        s.at_mass = e[i].mass;
        s.at_rank = e[i].rank;
        s.at_key = ~(uint32_t)(s.list[first + i] >> 32);
        s.at_index = (int)(uint32_t)s.list[first + i];
      }
    __syncthreads();
    const Place at{s.at_mass, s.at_rank, s.at_key, s.at_index};
    __syncthreads();
    return at;
  });
}

// A band of logits that holds a run of bins, widened by more than its roundings.
struct Band {
  float end, top;
};
__device__ __forceinline__ Band band_of(int lo, int hi, const Scale& c) {
  if (hi < lo) return Band{INFINITY, -INFINITY};
  const double slack = fabs(c.m) * 0x1p-40 + 1e-37;
  const double top = c.m - (double)lo / c.l64, end = c.m - (double)(hi + 1) / c.l64;
  return Band{(float)(end - fabs(end) * 0x1p-22 - slack),
              (float)(top + fabs(top) * 0x1p-22 + slack)};
}
// Puts the row's tokens of the bands on the list: those of the wanted bins and, now and
// then, a neighbour.  Most groups of 16 bytes have no logit as large as the lowest band's
// end.  (n_list counts what does not fit, too.)
template <int THREADS, int BANDS, bool F32>
__device__ __forceinline__ void gather(const Row<F32>& r, Lds& s, const Band (&band)[4]) {
  constexpr int E = Row<F32>::kE, U = 8;
  float least = band[0].end;
#pragma unroll
  for (int i = 1; i < BANDS; ++i) least = fminf(least, band[i].end);
  for (int at = (int)threadIdx.x; at < r.n_vec; at += U * THREADS) {
    u32x4 q[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int v = at + i * THREADS;
      q[i] = r.p[v < r.n_vec ? v : at];
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int v = at + i * THREADS;
      float z[E];
      logits_of<F32>(q[i], v < r.n_vec ? v : at, r.V, z);
      float m = z[0];
#pragma unroll
      for (int e = 1; e < E; ++e) m = fmaxf(m, z[e]);
      if (m >= least && v < r.n_vec) {
        bool in[E], any = false;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          in[e] = false;
#pragma unroll
          for (int k = 0; k < BANDS; ++k) in[e] |= (z[e] >= band[k].end) & (z[e] <= band[k].top);
          any |= in[e];
        }
        if (any) {
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (in[e]) {
              const uint32_t to = atomicAdd(&s.n_list, 1u);
              if (to < (uint32_t)kList)
                s.list[to] = (u64)(~key_of(z[e])) << 32 | (uint32_t)(v * E + e);
            }
        }
      }
    }
  }
}

// From the filled bins to the token, which thread 0 gets.
template <int THREADS, bool F32>
__device__ __noinline__ Drawn pick(Row<F32> r, Lds& s, Scale c, Settings g, Counts all) {
  constexpr int kPer = kBins / THREADS;
  {
    // cumulative masses and numbers
    double d[kPer], ds = 0, step = step_of((int)threadIdx.x * kPer, c);
    uint32_t n[kPer], ns = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = (int)threadIdx.x * kPer + i;
      const uint32_t k = s.num[b];
      d[i] = ds += (double)(s.mass[b] - k * kBias) * step;
      n[i] = ns += k;
      step *= 0.9892280131939755;        // 2^(-1 / 64)
    }
    double d0 = ds;
    uint32_t n0 = ns;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const double o_d = __shfl_up(d0, off);
      const uint32_t o_n = __shfl_up(n0, off);
      if ((int)(threadIdx.x % 64) >= off) {
        d0 += o_d;
        n0 += o_n;
      }
    }
    // The wave's part before this thread.  It is rounded along another path than the sum
    // that the threads before end with, so a bin without tokens would lie a rounding above
    // (or below) the one before it, and a target in between would find no token there.  A
    // thread therefore starts from the largest end of those before it: the masses never
    // fall, and rise at tokens only.  (Adding the waves before keeps equal ones equal.)
    const double up_d = __shfl_up(d0, 1);
    const uint32_t up_n = __shfl_up(n0, 1);
    d0 = threadIdx.x % 64 ? up_d : 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) d[i] += d0;
    double end = ns != 0 ? d[kPer - 1] : 0.0;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) end = fmax(end, __shfl_up(end, off));
    if (threadIdx.x % 64 == 63) {
      s.wave_d[threadIdx.x / 64] = end;
      s.wave_u[threadIdx.x / 64] = n0;
    }
    const double up_end = __shfl_up(end, 1);
    const double start = threadIdx.x % 64 ? up_end : 0.0;
    n0 = threadIdx.x % 64 ? up_n : 0u;
    __syncthreads();
    double w_d = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w)
      if (w < (int)(threadIdx.x / 64)) {
        w_d += s.wave_d[w];
        n0 += s.wave_u[w];
      }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      d[i] = w_d + (n[i] != 0 ? fmax(start, d[i]) : start);
      s.cum[threadIdx.x * kPer + i] = d[i];
      s.num[threadIdx.x * kPer + i] = n0 + n[i];
    }
    if (((int)threadIdx.x + 1) * kPer % 64 == 0) {
      s.group_cum[threadIdx.x * kPer / 64] = d[kPer - 1];
      s.group_num[threadIdx.x * kPer / 64] = n0 + n[kPer - 1];
    }
    if (threadIdx.x == 0) s.n_list = 0;
    __syncthreads();
  }
  const double total = s.cum[kBins - 1];
  const uint32_t near = s.num[kBins - 1], live = all.live;
  auto mass_before = [&](int b) { return b > 0 ? s.cum[b - 1] : 0.0; };
  auto num_before = [&](int b) { return b > 0 ? s.num[b - 1] : 0u; };

  // the bins of the targets, with bounds where a target is not known yet
  const double p = (double)g.top_p, u = (double)g.u;
  const uint32_t k1 = g.top_k > 0 && (uint32_t)g.top_k < live ? (uint32_t)g.top_k : live;
  const bool cut_k = k1 < near, cut_p = g.top_p < 1.0f;
  Wanted want;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    want.lo[i] = kBins;
    want.hi[i] = -1;
  }
  double m_lo = total, m_hi = total;
  uint32_t k_hi = k1;
  if (cut_k) {
    const int b = bin_of(s, Target{kCount, k1, 0.0}, near);
    want.lo[0] = want.hi[0] = b;
    m_lo = mass_before(b);
    m_hi = s.cum[b];
  }
  if (cut_p) {
    want.hi[1] = bin_of(s, Target{kReach, 0, p * m_hi}, near);
    want.lo[1] = cut_k ? bin_of(s, Target{kReach, 0, p * m_lo}, near) : want.hi[1];
    m_lo = fmin(m_lo, mass_before(want.lo[1]));
    m_hi = fmin(m_hi, s.cum[want.hi[1]]);
    k_hi = k_hi < s.num[want.hi[1]] ? k_hi : s.num[want.hi[1]];
  }
  const bool cut_m = all.min < k_hi && all.min < near;
  if (cut_m) {
    const int b = bin_of(s, Target{kCount, all.min, 0.0}, near);
    want.lo[2] = want.hi[2] = b;
    m_lo = fmin(m_lo, mass_before(b));
    m_hi = fmin(m_hi, s.cum[b]);
  }
  want.hi[3] = bin_of(s, Target{kExceed, 0, u * m_hi}, near);
  want.lo[3] = m_lo < m_hi ? bin_of(s, Target{kExceed, 0, u * m_lo}, near) : want.hi[3];
  const Cuts cuts{p, u, total, k1, all.min, near, cut_k, cut_p, cut_m};

  uint32_t n_want = 0;         // (a bin wanted twice counts twice)
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (want.hi[i] >= want.lo[i]) n_want += s.num[want.hi[i]] - num_before(want.lo[i]);

  uint32_t kept = k1;
  double M = total;
  Place at;
  if (__builtin_expect(n_want <= (uint32_t)kList, 1)) {
    Band bands[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) bands[i] = band_of(want.lo[3 - i], want.hi[3 - i], c);
    // (the draw's is first; of the cuts' often one is left)
    const int more = (int)cut_k + (int)cut_p + (int)cut_m;
    if (more == 1) bands[1] = cut_m ? bands[1] : cut_p ? bands[2] : bands[3];
    if (more == 0)
      gather<THREADS, 1>(r, s, bands);
    else if (more == 1)
      gather<THREADS, 2>(r, s, bands);
    else
      gather<THREADS, 4>(r, s, bands);
    __syncthreads();
  }
  const uint32_t n_list = s.n_list;
  if (__builtin_expect(n_want > (uint32_t)kList || n_list > (uint32_t)kList, 0)) {
    __syncthreads();
    at = one_by_one<THREADS>(r, s, c, cuts, &kept, &M);
  } else if (n_list <= 64) {
    if (threadIdx.x >= 64) return no_token();       // (the first wave has the result)
    at = resolve_short(s, c, cuts, want, (int)n_list, &kept, &M);
  } else {
    at = resolve_long<THREADS>(s, c, cuts, want, (int)n_list, &kept, &M);
  }
  if (all.min < kept) kept = all.min;        // (tokens past the bins that min_p drops)
  const double lw = -x_of(value_of(at.key), c) * (0.69314718055994530942 / 64.0);
  return Drawn{at.index, (float)(lw - log(total)), (float)(lw - log(M)), kept};
}

__device__ __forceinline__ void clear_bins(Lds& s, int threads) {
  for (int i = (int)threadIdx.x; i < kBins + kSpare; i += threads) {
    s.mass[i] = 0;
    s.num[i] = 0;
  }
}

// ------------------------------------------------------------------ a work-group per row
constexpr int kRowThreads = 512;

template <bool F32>
__global__ __launch_bounds__(kRowThreads, 4) void sample_rows_kernel(SampleArgs a, int64_t t0,
                                                                     double unit) {
  __shared__ Lds s;
  const int64_t t = t0 + blockIdx.x;
  const Settings g = settings_of(a, t);
  if (g.left_out) return put(a, t, left_out());
  if (!g.legal) return put(a, t, no_token());
  const Row<F32> r = row_of<F32>(a, t);
  clear_bins(s, kRowThreads);
  const Top top = top_part<kRowThreads>(r, 0, r.n_vec);
  const float m = reduce<kRowThreads>(top.m, reinterpret_cast<float*>(s.wave_u), max_or_nan);
  if (!(fabsf(m) < INFINITY)) return put(a, t, no_token());
  Counts n;
  n.live = (uint32_t)r.V - reduce<kRowThreads>(top.masked, s.wave_u, Add());
  const Scale c = scale_of(m, g.tau, unit);
  n.min = fill_bins<kRowThreads>(r, 0, r.n_vec, s, c, g.min_p);
  put(a, t, pick<kRowThreads>(r, s, c, g, n));
}

// ------------------------------------------------------------------ few rows, in pieces
// Three launches: the pieces' largest logits; their bins, added to the row's in the
// workspace; the token.
constexpr int kPieceThreads = 512, kPickThreads = 1024;
struct RowBins {
  u64 mass[kBins];
  uint32_t num[kBins];
  uint32_t min;
  uint32_t pad[63];
};
struct PieceArgs {
  SampleArgs a;
  double unit;
  int pieces, vecs;     // of a row; 16-byte vectors of a piece
  RowBins* rows;
  Top* top;             // [row][piece]
};

// (at most 64 pieces: one a lane)
__device__ __forceinline__ Top row_top(const PieceArgs& p, int64_t t) {
  const int lane = threadIdx.x & 63;
  Top x = p.top[t * p.pieces + (lane < p.pieces ? lane : 0)];
  if (lane >= p.pieces) x.masked = 0;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    x.m = max_or_nan(x.m, __shfl_xor(x.m, off));
    x.masked += __shfl_xor(x.masked, off);
  }
  return x;
}

template <bool F32>
__global__ __launch_bounds__(kPieceThreads) void piece_max_kernel(PieceArgs p) {
  __shared__ float lds[kMaxWaves];
  const int64_t t = blockIdx.x / p.pieces;
  const int i = blockIdx.x % p.pieces;
  // this piece's share of the row's bins, cleared for the next launch
  uint32_t* const words = reinterpret_cast<uint32_t*>(p.rows + t);
  constexpr int kWords = sizeof(RowBins) / 4;
  const int share = (kWords + p.pieces - 1) / p.pieces;
  for (int w = i * share + (int)threadIdx.x; w < kWords && w < (i + 1) * share; w += kPieceThreads)
    words[w] = 0;
  const Settings g = settings_of(p.a, t);
  if (g.left_out || !g.legal) return;
  const Row<F32> r = row_of<F32>(p.a, t);
  const int64_t v0 = (int64_t)i * p.vecs, v1 = v0 + p.vecs < r.n_vec ? v0 + p.vecs : r.n_vec;
  Top top = top_part<kPieceThreads>(r, (int)v0, (int)v1);
  top.m = reduce<kPieceThreads>(top.m, lds, max_or_nan);
  top.masked = reduce<kPieceThreads>(top.masked, reinterpret_cast<uint32_t*>(lds), Add());
  if (threadIdx.x == 0) p.top[blockIdx.x] = top;
}

template <bool F32>
__global__ __launch_bounds__(kPieceThreads) void piece_bins_kernel(PieceArgs p) {
  __shared__ Lds s;
  const int64_t t = blockIdx.x / p.pieces;
  const int i = blockIdx.x % p.pieces;
  const Settings g = settings_of(p.a, t);
  if (g.left_out || !g.legal) return;
  const float m = row_top(p, t).m;
  if (!(fabsf(m) < INFINITY)) return;
  clear_bins(s, kPieceThreads);
  __syncthreads();
  const Row<F32> r = row_of<F32>(p.a, t);
  const Scale c = scale_of(m, g.tau, p.unit);
  const int64_t v0 = (int64_t)i * p.vecs, v1 = v0 + p.vecs < r.n_vec ? v0 + p.vecs : r.n_vec;
  const uint32_t n_min = fill_bins<kPieceThreads>(r, (int)v0, (int)v1, s, c, g.min_p);
  RowBins& to = p.rows[t];
  for (int b = (int)threadIdx.x; b < kBins; b += kPieceThreads)
    if (s.num[b] != 0) {
      atomicAdd(&to.mass[b], s.mass[b]);
      atomicAdd(&to.num[b], s.num[b]);
    }
  if (threadIdx.x == 0 && n_min != kAll && n_min != 0) atomicAdd(&to.min, n_min);
}

template <bool F32>
__global__ __launch_bounds__(kPickThreads) void pick_kernel(PieceArgs p) {
  __shared__ Lds s;
  const int64_t t = blockIdx.x;
  const Settings g = settings_of(p.a, t);
  if (g.left_out) return put(p.a, t, left_out());
  if (!g.legal) return put(p.a, t, no_token());
  const Top top = row_top(p, t);
  if (!(fabsf(top.m) < INFINITY)) return put(p.a, t, no_token());
  const RowBins& from = p.rows[t];
#pragma unroll
  for (int i = 0; i < kBins / kPickThreads; ++i) {
    const int b = (int)threadIdx.x + i * kPickThreads;
    s.mass[b] = from.mass[b];
    s.num[b] = from.num[b];
  }
  const Counts n{(uint32_t)p.a.vocab - top.masked, g.min_p > 0.0f ? from.min : kAll};
  __syncthreads();
  put(p.a, t, pick<kPickThreads>(row_of<F32>(p.a, t), s, scale_of(top.m, g.tau, p.unit), g, n));
}

// Pieces of a row: about a work-group a CU in all (256), each of at least 512 vectors
// (clearing and adding up its bins costs a piece about as much), and at most 64; one: a
// work-group per row.
int pieces_of(int64_t n_tok, int64_t vocab) {
  const int64_t vecs = vocab / 8;
  int64_t most = vecs / 512, want = 256 / (n_tok > 0 ? n_tok : 1);
  if (want > most) want = most;
  if (want > 64) want = 64;
  return want < 2 ? 1 : (int)want;
}

}  // namespace

size_t sample_ws_bytes(int64_t n_tok, int64_t vocab) {
  const int pieces = pieces_of(n_tok, vocab);
  if (n_tok == 0 || pieces == 1) return 0;
  return (size_t)n_tok * sizeof(RowBins) +
         (size_t)round_up(n_tok * pieces * (int64_t)sizeof(Top), 256);
}

hipError_t launch_sample(const SampleArgs& a, bool f32, char* ws, hipStream_t s) {
  // a bin's sum of `vocab` integers up to 2^bits stays below 2^63
  int bits = 45;
  while (bits > 32 && ((double)a.vocab * exp2((double)bits)) > 0x1p63) --bits;
  const double unit = exp2((double)bits);
  const int pieces = pieces_of(a.n_tok, a.vocab);
  if (pieces == 1) {
    auto kernel = f32 ? sample_rows_kernel<true> : sample_rows_kernel<false>;
    constexpr int64_t kMost = 1 << 22;      // rows of a launch (2^31 threads)
    for (int64_t t = 0; t < a.n_tok; t += kMost)
      hipLaunchKernelGGL(kernel, dim3((unsigned)(a.n_tok - t < kMost ? a.n_tok - t : kMost)),
                         dim3(kRowThreads), 0, s, a, t, unit);
    return hipGetLastError();
  }
  const int e = f32 ? 4 : 8;
  const int64_t n_vec = ((int64_t)a.vocab + e - 1) / e;
  PieceArgs p{a, unit, pieces, (int)((n_vec + pieces - 1) / pieces),
              reinterpret_cast<RowBins*>(ws),
              reinterpret_cast<Top*>(ws + (size_t)a.n_tok * sizeof(RowBins))};
  const dim3 grid((unsigned)(a.n_tok * pieces));
  if (f32) {
    hipLaunchKernelGGL(piece_max_kernel<true>, grid, dim3(kPieceThreads), 0, s, p);
    hipLaunchKernelGGL(piece_bins_kernel<true>, grid, dim3(kPieceThreads), 0, s, p);
    hipLaunchKernelGGL(pick_kernel<true>, dim3((unsigned)a.n_tok), dim3(kPickThreads), 0, s, p);
  } else {
    hipLaunchKernelGGL(piece_max_kernel<false>, grid, dim3(kPieceThreads), 0, s, p);
    hipLaunchKernelGGL(piece_bins_kernel<false>, grid, dim3(kPieceThreads), 0, s, p);
    hipLaunchKernelGGL(pick_kernel<false>, dim3((unsigned)a.n_tok), dim3(kPickThreads), 0, s, p);
  }
  return hipGetLastError();
}

}  // namespace logra
