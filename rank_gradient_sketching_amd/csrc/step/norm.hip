// logra_grad_norm, logra_grad_clip: the norm of many gradients taken as one
// vector, the factor that clips it, and the clipped gradients, on gfx950.
//
// Mathematics.  norm = |s| sqrt(sum g^2), scale = s min(1, max_norm / norm).  A
// square and its sum are one fp64 fused step per entry: the largest fp32 squares
// to 1e77 and the smallest to 1e-90, so neither end needs a second pass or a
// running scale, and the sum carries 2^-53 of each term.  fp64 costs nothing here
// (a conversion and a fused step per entry, 64 entries in 8 cycles of a SIMD: the
// chip does 2 10^13 entries a second and the HBM brings 3 10^12).  The largest
// magnitude is an integer maximum of the bits without the sign, which puts NaN
// above infinity.
//
// A work-group takes consecutive entries of one tensor and leaves one partial sum;
// a second launch adds them, in a fixed order, for all tensors and for each.  A
// work-group finds its tensor by bisecting the table's first work-groups (the same
// cache lines for all).  Bound: HBM bytes.  233570304 bf16 entries take 73 us, 6.4 TB/s,
// with loads past the caches (ordinary ones: 16 % more).  Tensors off 16 bytes are read entry
// by entry: 64 Mi fp32 84 us instead of 43, bf16 79 instead of 23 (their clip in place 81
// instead of 83, and 50 instead of 48).
#include <math.h>

#include "common.hpp"
#include "internal.hpp"
#include "step/internal_step.hpp"

namespace logra {

namespace {

typedef unsigned long long u64;

constexpr int kThreads = 256;
constexpr int kLoads = 8;                 // 16-byte loads in flight per lane
constexpr int kBytes = 16 * kThreads * kLoads;   // of one step
// Work-groups in all, about: past it a work-group takes more steps.  (2048 to 16384 with
// four loads or eight: within 2 %.)
constexpr int64_t kGroups = 4096;

int64_t elem(bool f32) { return f32 ? 4 : 2; }

// The tensor of work-group b: the last one whose first work-group is <= b.
__device__ __forceinline__ int find_item(const int32_t* __restrict__ first, int n, int b) {
  int lo = 0, hi = n;          // first[lo] <= b < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= b)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void unpack(const u32x4& v, bool f32, float* x) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    if (f32) {
      x[p] = __uint_as_float(v[p]);
    } else {
      x[2 * p] = bf16_lo(v[p]);
      x[2 * p + 1] = bf16_hi(v[p]);
    }
  }
}

template <bool INF>
__device__ __forceinline__ void add(double& acc, float x) {
  if constexpr (INF) {
    // (a NaN's pattern is the largest; kept in the low word of the accumulator)
    const uint32_t m = __float_as_uint(x) & 0x7FFFFFFFu;
    const uint32_t o = (uint32_t)__double_as_longlong(acc);
    acc = __longlong_as_double((long long)(m > o ? m : o));
  } else {
    acc = fma((double)x, (double)x, acc);
  }
}
template <bool INF>
__device__ __forceinline__ double join(double a, double b) {
  if constexpr (INF) {
    const u64 x = (u64)__double_as_longlong(a), y = (u64)__double_as_longlong(b);
    return __longlong_as_double((long long)(x > y ? x : y));
  } else {
    return a + b;
  }
}
// Sum (or maximum) over the work-group's threads, in thread 0.
template <bool INF, int THREADS>
__device__ __forceinline__ double join_all(double acc, double* lds) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) acc = join<INF>(acc, __shfl_xor(acc, off));
  const int w = threadIdx.x / 64;
  if (threadIdx.x % 64 == 0) lds[w] = acc;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int i = 1; i < THREADS / 64; ++i) acc = join<INF>(acc, lds[i]);
  return acc;
}

template <bool INF, bool F32>
__device__ __forceinline__ double chunk_sum(const void* g, int64_t at, int64_t end,
                                            bool vec) {
  constexpr int E = F32 ? 4 : 8;
  double acc[4] = {0, 0, 0, 0};
  if (vec) {
    const u32x4* const src = static_cast<const u32x4*>(g);
    for (; at + E * kThreads * kLoads <= end; at += E * kThreads * kLoads) {
      u32x4 v[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        v[i] = __builtin_nontemporal_load(src + at / E + i * kThreads + threadIdx.x);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        float x[8];
        unpack(v[i], F32, x);
#pragma unroll
        for (int e = 0; e < E; ++e) add<INF>(acc[e & 3], x[e]);
      }
    }
    if (at + E <= end) {      // the last, incomplete step: zeros past the end
      u32x4 v[kLoads];
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int64_t i = at + ((int64_t)k * kThreads + threadIdx.x) * E;
        v[k] = u32x4{0, 0, 0, 0};
        if (i + E <= end) v[k] = __builtin_nontemporal_load(src + i / E);
      }
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        float x[8];
        unpack(v[k], F32, x);
#pragma unroll
        for (int e = 0; e < E; ++e) add<INF>(acc[e & 3], x[e]);
      }
    }
    at = end / E * E;      // entries of the last, incomplete 16 bytes
  }
  for (int64_t i = at + threadIdx.x; i < end; i += kThreads)
    add<INF>(acc[0], F32 ? static_cast<const float*>(g)[i]
                         : bf16_to_f32(static_cast<const uint16_t*>(g)[i]));
  return join<INF>(join<INF>(acc[0], acc[1]), join<INF>(acc[2], acc[3]));
}

// Entries [at, end) of its tensor that a work-group takes.
__device__ __forceinline__ void my_range(const GradItem& q, int b, int first, int loops,
                                         int64_t* at, int64_t* end) {
  const int64_t chunk = (int64_t)loops * kBytes / (q.g_f32 ? 4 : 2);
  *at = (int64_t)(b - first) * chunk;
  *end = *at + chunk < q.n ? *at + chunk : q.n;
}

template <bool INF>
__global__ __launch_bounds__(kThreads) void norm_partial_kernel(const GradItem* __restrict__ items,
                                                                const int32_t* __restrict__ first,
                                                                int n, int loops,
                                                                double* __restrict__ partial) {
  __shared__ double lds[kThreads / 64];
  const int b = (int)blockIdx.x;
  const int i = find_item(first, n, b);
  const GradItem q = items[i];
  int64_t at, end;
  my_range(q, b, first[i], loops, &at, &end);
  const double part = q.g_f32 ? chunk_sum<INF, true>(q.g, at, end, q.vec)
                              : chunk_sum<INF, false>(q.g, at, end, q.vec);
  const double all = join_all<INF, kThreads>(part, lds);
  if (threadIdx.x == 0) partial[b] = all;
}

// Work-group 0 joins all partial sums into norm and scale, work-group 1 + i those of
// tensor i.
template <bool INF>
__global__ __launch_bounds__(1024) void norm_join_kernel(GradNormArgs a,
                                                         const double* __restrict__ partial) {
  __shared__ double lds[16];
  const int i = (int)blockIdx.x - 1;
  const bool every = i < 0 || a.groups == 0;   // (no entries at all: no table to read)
  const int lo = every ? 0 : a.first[i], hi = every ? a.groups : a.first[i + 1];
  double acc = 0;
  for (int b = lo + (int)threadIdx.x; b < hi; b += 1024) acc = join<INF>(acc, partial[b]);
  acc = join_all<INF, 1024>(acc, lds);
  if (threadIdx.x != 0) return;
  if constexpr (INF) acc = (double)__uint_as_float((uint32_t)__double_as_longlong(acc));
  const double s = a.grad_scale != nullptr ? (double)a.grad_scale[0] : 1.0;
  const double norm = fabs(s) * (INF ? acc : sqrt(acc));
  if (i >= 0) {
    a.norms[i] = (float)norm;
    return;
  }
  if (a.norm != nullptr) a.norm[0] = (float)norm;
  if (a.scale != nullptr)
    a.scale[0] = (float)(norm != norm ? norm : norm > a.max_norm ? s * (a.max_norm / norm) : s);
}

__device__ __forceinline__ void store_scaled(void* out, bool f32, int64_t i, float x) {
  if (f32)
    static_cast<float*>(out)[i] = x;
  else
    static_cast<uint16_t*>(out)[i] = f32_to_bf16(x);
}

template <bool PAST, class T>
__device__ __forceinline__ T load_as(const T* p) {
  if constexpr (PAST) return __builtin_nontemporal_load(p);
  return *p;
}
template <bool PAST, class T>
__device__ __forceinline__ void store_as(T x, T* p) {
  if constexpr (PAST)
    __builtin_nontemporal_store(x, p);
  else
    *p = x;
}

// PAST: past the caches.
template <bool PAST, bool GF32, bool OF32>
__device__ __forceinline__ void clip_chunk(const void* g, void* out, int64_t at, int64_t end,
                                           bool vec, float scale) {
  constexpr int E = GF32 ? 4 : 8;
  if (vec) {
    const u32x4* const src = static_cast<const u32x4*>(g);
    for (; at + E <= end; at += E * kThreads * kLoads) {
      u32x4 v[kLoads];
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int64_t i = at + ((int64_t)k * kThreads + threadIdx.x) * E;
        if (i + E <= end) v[k] = load_as<PAST>(src + i / E);
      }
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int64_t i = at + ((int64_t)k * kThreads + threadIdx.x) * E;
        if (i + E > end) continue;
        float x[8];
        unpack(v[k], GF32, x);
        if constexpr (OF32) {
          f32x4* const dst = reinterpret_cast<f32x4*>(static_cast<float*>(out) + i);
#pragma unroll
          for (int e = 0; e < E; e += 4)
            store_as<PAST>(
                f32x4{x[e] * scale, x[e + 1] * scale, x[e + 2] * scale, x[e + 3] * scale},
                dst + e / 4);
        } else if constexpr (GF32) {
          const uint32_t lo = pack_bf16x2(x[0] * scale, x[1] * scale);
          const uint32_t hi = pack_bf16x2(x[2] * scale, x[3] * scale);
          store_as<PAST>(u32x2{lo, hi},
                         reinterpret_cast<u32x2*>(static_cast<uint16_t*>(out) + i));
        } else {
          u32x4 y;
#pragma unroll
          for (int p = 0; p < 4; ++p) y[p] = pack_bf16x2(x[2 * p] * scale, x[2 * p + 1] * scale);
          store_as<PAST>(y, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + i));
        }
      }
    }
    at = end / E * E;
  }
  for (int64_t i = at + threadIdx.x; i < end; i += kThreads)
    store_scaled(out, OF32, i,
                 scale * (GF32 ? static_cast<const float*>(g)[i]
                               : bf16_to_f32(static_cast<const uint16_t*>(g)[i])));
}

template <bool PAST>
__global__ __launch_bounds__(kThreads) void clip_kernel(const GradItem* __restrict__ items,
                                                        const int32_t* __restrict__ first, int n,
                                                        int loops,
                                                        const float* __restrict__ scale_p) {
  const float scale = scale_p[0];
  const int b = (int)blockIdx.x;
  const int i = find_item(first, n, b);
  const GradItem q = items[i];
  // a factor of one leaves an array that is written in place as it is
  if (scale == 1.0f && q.out == q.g) return;
  int64_t at, end;
  my_range(q, b, first[i], loops, &at, &end);
  if (q.g_f32) {
    if (q.out_f32)
      clip_chunk<PAST, true, true>(q.g, q.out, at, end, q.vec, scale);
    else
      clip_chunk<PAST, true, false>(q.g, q.out, at, end, q.vec, scale);
  } else {
    if (q.out_f32)
      clip_chunk<PAST, false, true>(q.g, q.out, at, end, q.vec, scale);
    else
      clip_chunk<PAST, false, false>(q.g, q.out, at, end, q.vec, scale);
  }
}

// Past the caches from 128 MiB of gradients: norm and clip of 233570304 bf16 entries 250
// us (268 through them), 4 x 4096 x 4096 fp32 in place 152 (158); 168 x 13001 bf16, which
// the caches hold, 14.2 (11.1), 5000 x 1536 fp32 in place 33.9 (32.5).
constexpr int64_t kLargeBytes = (int64_t)128 << 20;

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

bool grad_lay_out(GradTable* head, GradItem* items, int32_t* first) {
  int64_t steps = 0, bytes = 0;
  for (int i = 0; i < head->n; ++i) {
    steps += (items[i].n * elem(items[i].g_f32) + kBytes - 1) / kBytes;
    bytes += items[i].n * elem(items[i].g_f32);
  }
  head->large = bytes >= kLargeBytes;
  const int64_t loops = (steps + kGroups - 1) / kGroups;
  head->loops = (int32_t)(loops < 1 ? 1 : loops > (1 << 20) ? 1 << 20 : loops);
  int64_t groups = 0;
  for (int i = 0; i < head->n; ++i) {
    GradItem& q = items[i];
    q.vec = on16(q.g) && on16(q.out);
    first[i] = (int32_t)groups;
    const int64_t chunk = (int64_t)head->loops * kBytes / elem(q.g_f32);
    groups += (q.n + chunk - 1) / chunk;
    if (groups >= (int64_t(1) << 24)) return false;   // 2^32 threads
  }
  first[head->n] = (int32_t)groups;
  head->groups = (int32_t)groups;
  return true;
}

hipError_t launch_grad_norm(const GradNormArgs& a, double* partial, hipStream_t s) {
  if (a.groups > 0) {
    if (a.inf_norm)
      hipLaunchKernelGGL((norm_partial_kernel<true>), dim3((unsigned)a.groups), dim3(kThreads), 0,
                         s, a.items, a.first, a.n, a.loops, partial);
    else
      hipLaunchKernelGGL((norm_partial_kernel<false>), dim3((unsigned)a.groups), dim3(kThreads), 0,
                         s, a.items, a.first, a.n, a.loops, partial);
  }
  const dim3 grid(1u + (a.norms != nullptr ? (unsigned)a.n : 0u));
  if (a.inf_norm)
    hipLaunchKernelGGL((norm_join_kernel<true>), grid, dim3(1024), 0, s, a, partial);
  else
    hipLaunchKernelGGL((norm_join_kernel<false>), grid, dim3(1024), 0, s, a, partial);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const GradNormArgs& a, const float* scale, hipStream_t s) {
  hipLaunchKernelGGL(a.large ? clip_kernel<true> : clip_kernel<false>, dim3((unsigned)a.groups),
                     dim3(kThreads), 0, s, a.items, a.first, a.n, a.loops, scale);
  return hipGetLastError();
}

}  // namespace logra
