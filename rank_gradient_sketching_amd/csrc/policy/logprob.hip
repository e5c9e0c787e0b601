// logra_token_logprob and its gradient, on gfx950: log probabilities of given
// tokens under softmax(z / tau), the entropy of that distribution and its most
// probable tokens, in one pass over the logits.
//
// Mathematics.  With m the largest logit of a row, d_j = (z_j - m) log2(e) / tau
// and w_j = 2^d_j, a row needs s = sum w and u = sum w d:
//   lse = m / tau + ln s,   logp = (z_target - m) / tau - ln s,
//   H = ln s - ln(2) u / s  (both terms >= 0: no cancellation).
// Each thread keeps (m, s, u) about its own running maximum (a rescale when a
// group of its elements raises it), the states of a wave meet in a butterfly
// and those of a row's waves in LDS, always in the same order.  m is
// subtracted from the unscaled logit, which is exact for the tokens that carry
// weight, so the exponent's rounding is relative to d and not to z / tau.
// Masked tokens: z = -inf gives w = 0; d is clamped at kLow in u alone, so that
// 0 * -inf does not arise while NaN (and +inf, which becomes NaN) still reach
// s.  m starts at the lowest finite float instead of -inf: no case of its own
// for a thread that has seen nothing yet.
//
// Alternatives.  Value and index of a token make one 64-bit key (the float's
// bits in an order-preserving form above the inverted index), so "larger
// logit, then lower index" is one integer comparison and keys are distinct:
// the result does not depend on the order of anything.  A wave keeps its 64
// best keys sorted over its lanes.  A group of elements is looked at closer
// only when its largest value (already at hand for the softmax) beats the
// n_top-th key's; passing elements are collected in LDS, and 64 of them at a
// time are sorted by a bitonic network and merged in.  On a wave's first group
// each lane first offers its own maximum: one sort then gives a threshold that
// nearly all other elements fail.
//
// Bound: the stream of the logits.  One work-group per row where the rows
// fill the chip; fewer rows are cut into pieces whose states and keys a second
// kernel joins.
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
constexpr float kMinFloat = -3.4028234663852886e38f;

// ---------------------------------------------------------------- softmax states
struct State {
  float m, s, u;
};

__device__ __forceinline__ State merge_states(const State& a, const State& b, float l2t) {
  const float M = fmaxf(a.m, b.m);
  const float da = fmaxf((a.m - M) * l2t, kLow);
  const float db = fmaxf((b.m - M) * l2t, kLow);
  const float fa = exp2_normal(da), fb = exp2_normal(db);
  State o;
  o.m = M;
  o.s = fa * a.s + fb * b.s;
  o.u = fa * fmaf(a.s, da, a.u) + fb * fmaf(b.s, db, b.u);
  return o;
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

// Adds G elements whose maximum is gmax (-inf where there is none).
template <int G>
__device__ __forceinline__ void add_group(State& st, const float* z, float gmax, float l2t) {
  if (gmax > st.m) {
    const float dm = fmaxf((st.m - gmax) * l2t, kLow);
    const float f = exp2_normal(dm);
    st.u = f * fmaf(st.s, dm, st.u);
    st.s *= f;
    st.m = gmax;
  }
#pragma unroll
  for (int e = 0; e < G; ++e) {
    const float d = (z[e] - st.m) * l2t;
    const float w = exp2_normal(d);
    st.s += w;
    st.u = fmaf(w, fmaxf(d, kLow), st.u);
  }
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

__device__ __forceinline__ u64 shfl_xor64(u64 x, int mask) {
  const uint32_t lo = __shfl_xor((uint32_t)x, mask);
  const uint32_t hi = __shfl_xor((uint32_t)(x >> 32), mask);
  return ((u64)hi << 32) | lo;
}
__device__ __forceinline__ u64 compare_exchange(u64 x, int j, bool keep_max) {
  const u64 y = shfl_xor64(x, j);
  return (x > y) == keep_max ? x : y;
}

// A wave's best 64 keys, lane i the i-th (0: none).
struct BestKeys {
  u64 best;
  u64 thr_key;   // the n_top-th best key so far
  float thr;     // its value (-inf while there is none)
  int count;     // keys waiting in buf (below 64 between calls)
  u64* buf;      // this wave's 128 places in LDS
};

__device__ __forceinline__ BestKeys no_keys(u64* buf) {
  return BestKeys{0, 0, -INFINITY, 0, buf};
}

// Merges 64 more keys (0: none), one per lane.
__device__ __forceinline__ void merge_keys(BestKeys& b, u64 x, int n_top) {
  const int lane = threadIdx.x & 63;
  // ascending bitonic sort
#pragma unroll
  for (int k = 2; k <= 64; k <<= 1) {
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1)
      x = compare_exchange(x, j, ((lane & j) == 0) != ((lane & k) == 0));
  }
  // descending against ascending: the larger of each pair are the best 64
  b.best = b.best > x ? b.best : x;
#pragma unroll
  for (int j = 32; j > 0; j >>= 1) b.best = compare_exchange(b.best, j, (lane & j) == 0);
  const uint32_t lo = __shfl((uint32_t)b.best, n_top - 1);
  const uint32_t hi = __shfl((uint32_t)(b.best >> 32), n_top - 1);
  b.thr_key = ((u64)hi << 32) | lo;
  b.thr = b.thr_key ? key_value(b.thr_key) : -INFINITY;
}

__device__ __forceinline__ void flush_keys(BestKeys& b, int n_top) {
  const int lane = threadIdx.x & 63;
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  const u64 x = lane < b.count ? b.buf[lane] : 0;
  const bool more = 64 + lane < b.count;
  const u64 y = more ? b.buf[64 + lane] : 0;
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  if (more) b.buf[lane] = y;
  b.count = b.count > 64 ? b.count - 64 : 0;
  merge_keys(b, x, n_top);
}

// One element per lane (every lane of the wave calls this).
__device__ __forceinline__ void offer(BestKeys& b, float x, uint32_t idx, bool take, int n_top) {
  const u64 key = order_key(x, idx);
  const bool pass = take && x > -INFINITY && key > b.thr_key;
  const u64 mask = __ballot(pass);
  if (mask == 0) return;
  const int lane = threadIdx.x & 63;
  if (pass) b.buf[b.count + __popcll(mask & ((u64(1) << lane) - 1))] = key;
  b.count += __popcll(mask);
  if (b.count >= 64) flush_keys(b, n_top);
}

// A group of G elements per lane from index idx; gmax its maximum.
template <int G>
__device__ __forceinline__ void offer_group(BestKeys& b, const float* z, float gmax, uint32_t idx,
                                            bool first, int n_top) {
  int own = -1;   // the element already offered
  if (first) {
    // (the first of equal maxima, so the one with the lowest index)
#pragma unroll
    for (int e = G - 1; e >= 0; --e) own = z[e] == gmax ? e : own;
    offer(b, gmax, idx + (uint32_t)(own < 0 ? 0 : own), own >= 0, n_top);
    if (b.count > 0) flush_keys(b, n_top);
  }
  // Elements of later groups have larger indices than all before them, so an
  // equal value does not pass; inside a group the keys decide.
  if (__ballot(first ? gmax > -INFINITY : gmax > b.thr) == 0) return;
#pragma unroll
  for (int e = 0; e < G; ++e) offer(b, z[e], idx + e, e != own, n_top);
}

// ---------------------------------------------------------------- loads
// The 16-byte group at column `col`; columns past V read as -inf.
template <class T>
struct Group;
template <>
struct Group<uint16_t> {
  static constexpr int G = 8;
  static __device__ __forceinline__ void load(const uint16_t* row, int64_t col, int V, float* z) {
    if (col + G <= V) {
      const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row + col));
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        z[2 * p] = bf16_lo(v[p]);
        z[2 * p + 1] = bf16_hi(v[p]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < G; ++e) z[e] = col + e < V ? bf16_to_f32(row[col + e]) : -INFINITY;
    }
  }
  static __device__ __forceinline__ void store(uint16_t* row, int64_t col, int V, const float* z) {
    if (col + G <= V) {
      u32x4 v;
#pragma unroll
      for (int p = 0; p < 4; ++p) v[p] = pack_bf16x2(z[2 * p], z[2 * p + 1]);
      __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(row + col));
    } else {
#pragma unroll
      for (int e = 0; e < G; ++e)
        if (col + e < V) row[col + e] = f32_to_bf16(z[e]);
    }
  }
  static __device__ __forceinline__ float one(const uint16_t* row, int64_t col) {
    return bf16_to_f32(row[col]);
  }
};
template <>
struct Group<float> {
  static constexpr int G = 4;
  static __device__ __forceinline__ void load(const float* row, int64_t col, int V, float* z) {
    if (col + G <= V) {
      const f32x4 v = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(row + col));
#pragma unroll
      for (int e = 0; e < G; ++e) z[e] = v[e];
    } else {
#pragma unroll
      for (int e = 0; e < G; ++e) z[e] = col + e < V ? row[col + e] : -INFINITY;
    }
  }
  static __device__ __forceinline__ void store(float* row, int64_t col, int V, const float* z) {
    if (col + G <= V) {
      const f32x4 v = {z[0], z[1], z[2], z[3]};
      __builtin_nontemporal_store(v, reinterpret_cast<f32x4*>(row + col));
    } else {
#pragma unroll
      for (int e = 0; e < G; ++e)
        if (col + e < V) row[col + e] = z[e];
    }
  }
  static __device__ __forceinline__ float one(const float* row, int64_t col) { return row[col]; }
};

// ---------------------------------------------------------------- results of a row
__device__ __forceinline__ bool left_out(const LogprobArgs& a, int64_t row) {
  if (a.target == nullptr) return false;
  const int64_t t = a.target[row];
  return t < 0 || t >= a.vocab;
}

// By one thread of the row.
template <class T>
__device__ __forceinline__ void write_row(const LogprobArgs& a, int64_t row, const State& st) {
  const float inv_tau = 1.0f / a.tau;
  const float ln_s = logf(st.s);
  if (a.lse) a.lse[row] = st.m / a.tau + ln_s;
  if (a.entropy) a.entropy[row] = ln_s - kLn2 * (st.u / st.s);
  if (a.logp) {
    const float zt =
        Group<T>::one(static_cast<const T*>(a.z) + row * a.ld, a.target[row]);
    a.logp[row] = (zt - st.m) * inv_tau - ln_s;
  }
}
// By the lanes of one wave of the row.
__device__ __forceinline__ void write_keys(const LogprobArgs& a, int64_t row, const State& st,
                                           u64 key) {
  const int lane = threadIdx.x & 63;
  if (lane >= a.n_top) return;
  a.top_idx[row * a.n_top + lane] = key ? key_index(key) : -1;
  a.top_logp[row * a.n_top + lane] =
      key ? (key_value(key) - st.m) * (1.0f / a.tau) - logf(st.s) : -INFINITY;
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
  constexpr int G = Group<T>::G;
  __shared__ State wst[kWaves];
  __shared__ u64 wbuf[TOP ? kWaves * 128 : 1];
  const int wave = threadIdx.x >> 6;
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
    BestKeys bk = no_keys(wbuf + (TOP ? wave * 128 : 0));
    bool first = true;
    // (whole waves stay in the loop: a wave's first column decides)
    for (int64_t c = c0 + (int64_t)wave * 64 * G; c < c1; c += (int64_t)kThreads * G) {
      const int64_t col = c + lane * G;
      float v[G];
      Group<T>::load(z, col < c1 ? col : c1, (int)c1, v);
      float gmax = v[0];
#pragma unroll
      for (int e = 1; e < G; ++e) gmax = fmaxf(gmax, v[e]);
      add_group<G>(st, v, gmax, l2t);
      if constexpr (TOP) {
        offer_group<G>(bk, v, gmax, (uint32_t)col, first, a.n_top);
        first = false;
      }
    }
    st = wave_state(st, l2t);
    if constexpr (TOP) {
      if (bk.count > 0) flush_keys(bk, a.n_top);
    }
    if (lane == 0) wst[wave] = st;
    if constexpr (TOP) wbuf[wave * 128 + lane] = bk.best;
    __syncthreads();
    if (wave == 0) {
      State t = wst[0];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) t = merge_states(t, wst[w], l2t);
      if constexpr (TOP) {
#pragma unroll 1
        for (int w = 1; w < kWaves; ++w) merge_keys(bk, wbuf[w * 128 + lane], a.n_top);
      }
      if (n_split == 1) {
        if (lane == 0) write_row<T>(a, row, t);
        if constexpr (TOP) write_keys(a, row, t, bk.best);
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
  __shared__ u64 buf[TOP ? 128 : 1];
  const int lane = threadIdx.x;
  const float l2t = kLog2e / a.tau;
  for (int64_t row = blockIdx.x; row < a.n_tok; row += gridDim.x) {
    if (left_out(a, row)) continue;
    State st{kMinFloat, 0.0f, 0.0f};
    for (int i = lane; i < n_split; i += 64) {
      const float* q = states + 3 * (row * n_split + i);
      st = merge_states(st, State{q[0], q[1], q[2]}, l2t);
    }
    st = wave_state(st, l2t);
    if (lane == 0) write_row<T>(a, row, st);
    if constexpr (TOP) {
      BestKeys bk = no_keys(buf);
      const int n = n_split * a.n_top;
      const u64* q = keys + row * n;
      for (int i = 0; i < n; i += 64) {
        const u64 x = i + lane < n ? q[i + lane] : 0;
        if (__ballot(x > bk.thr_key) != 0) merge_keys(bk, x, a.n_top);
      }
      write_keys(a, row, st, bk.best);
    }
  }
}

// dz over pieces of kGradGroups groups per thread.
constexpr int kGradGroups = 4;

template <class T>
__global__ __launch_bounds__(kThreads) void logprob_grad_kernel(LogprobGradArgs a, int n_pieces) {
  constexpr int G = Group<T>::G;
  constexpr int64_t kPiece = (int64_t)kThreads * G * kGradGroups;
  const int64_t n_tasks = a.n_tok * n_pieces;
  // 1 / tau as two floats: z / tau keeps fp32 accuracy in one fused step
  const float ih = 1.0f / a.tau;
  const float il = fmaf(-a.tau, ih, 1.0f) / a.tau;
  for (int64_t task = blockIdx.x; task < n_tasks; task += gridDim.x) {
    const int64_t row = task / n_pieces;
    const int64_t c0 = (task - row * n_pieces) * kPiece;
    const T* z = static_cast<const T*>(a.z) + row * a.ld;
    T* dz = static_cast<T*>(a.dz) + row * a.ldz;
    const int64_t target = a.target ? a.target[row] : -1;
    if (a.target && (target < 0 || target >= a.vocab)) {
      const float zero[G] = {};
#pragma unroll
      for (int i = 0; i < kGradGroups; ++i) {
        const int64_t col = c0 + ((int64_t)i * kThreads + threadIdx.x) * G;
        if (col < a.vocab) Group<T>::store(dz, col, a.vocab, zero);
      }
      continue;
    }
    const float lse = a.lse[row];
    const float g = a.d_logp ? a.d_logp[row] : 0.0f;
    const float gl = a.d_lse ? a.d_lse[row] : 0.0f;
    const float gh = a.d_entropy ? a.d_entropy[row] : 0.0f;
    const float H = a.d_entropy ? a.entropy[row] : 0.0f;
    // dz_j = p_j (k0 + k1 log p_j) + [j = target] kt
    const float k0 = (gl - g - gh * H) * ih, k1 = -gh * ih, kt = g * ih;
    float v[kGradGroups][G];
#pragma unroll
    for (int i = 0; i < kGradGroups; ++i) {
      const int64_t col = c0 + ((int64_t)i * kThreads + threadIdx.x) * G;
      if (col < a.vocab) Group<T>::load(z, col, a.vocab, v[i]);
    }
#pragma unroll
    for (int i = 0; i < kGradGroups; ++i) {
      const int64_t col = c0 + ((int64_t)i * kThreads + threadIdx.x) * G;
      if (col >= a.vocab) continue;
#pragma unroll
      for (int e = 0; e < G; ++e) {
        const float lp = fmaf(v[i][e], ih, fmaf(v[i][e] == -INFINITY ? 0.0f : v[i][e], il, -lse));
        const float p = exp2_normal(lp * kLog2e);
        // (a masked token: p = 0 and log p kept finite)
        float o = p * fmaf(k1, fmaxf(lp, kLow), k0);
        if (col + e == target) o += kt;
        v[i][e] = o;
      }
      Group<T>::store(dz, col, a.vocab, v[i]);
    }
  }
}

// Work-groups a chip full of streaming work wants, and the most a launch takes
// (tasks beyond it are walked by the same work-groups).
constexpr int64_t kFill = 1024;
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
  constexpr int64_t kPiece = (int64_t)kThreads * Group<T>::G * kGradGroups;
  const int n_pieces = (int)((a.vocab + kPiece - 1) / kPiece);
  const int64_t tasks = a.n_tok * n_pieces;
  hipLaunchKernelGGL((logprob_grad_kernel<T>), dim3((unsigned)(tasks < kMaxGrid ? tasks : kMaxGrid)),
                     dim3(kThreads), 0, s, a, n_pieces);
  return hipGetLastError();
}

}  // namespace

LogprobPlan make_logprob_plan(int64_t n_tok, int64_t vocab, int n_top) {
  LogprobPlan p{};
  // whole steps of a bf16 work-group (2048 columns) per piece, and no more
  // pieces than fill the chip
  constexpr int64_t kStep = (int64_t)kThreads * 8;
  const int64_t steps = (vocab + kStep - 1) / kStep;
  int64_t want = n_tok > 0 ? (kFill + n_tok - 1) / n_tok : 1;
  if (want > steps) want = steps;
  if (want < 1) want = 1;
  const int64_t per = (steps + want - 1) / want;
  p.piece = per * kStep;
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
