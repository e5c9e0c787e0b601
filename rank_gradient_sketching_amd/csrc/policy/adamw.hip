// logra_adamw_step: one AdamW step over many tensors, states in fp32 or in 8
// bits, on gfx950; logra_adamw_state_values: 8-bit states as values.
//
// Mathematics (per entry, fp32):
//   m' = b1 m + (1 - b1) g,   v' = b2 v + (1 - b2) g^2,
//   w' = w - lr ((m' / bc1) / (sqrt(v' / bc2) + eps) + wd w),
// written with r = sqrt(v'): sqrt(v' / bc2) = r / sqrt(bc2), so the 8-bit form,
// which holds r, needs no second root.
//
// The 8-bit form (include/logra_policy.h has its bits): 32 entries share an
// exponent byte, an entry is a small float below the block's largest, so
// decoding is a shift and an add on the fp32 pattern and no table is read.
// r is held instead of v because it needs half the binades.  Rounding adds a
// dither from a counter and truncates: rounded to nearest, v with beta2 =
// 0.999 would never move (the root changes by at most 0.05 % a step, the
// spacing is 3 to 6 %) - simulated over 6000 steps of unit-variance gradients,
// sqrt(v) then ended at 0.52 of its true value, and with the dither at 1.00
// with a spread of 0.09 (the counter's equally spaced dithers; 0.10 with
// random ones).  The m of a block share the 32 lanes' maximum by three
// cross-lane steps (four entries per lane, eight lanes per block).
//
// Bound: HBM bytes (a bf16 weight with fp32 master, bf16 gradient and fp32
// states moves 28 bytes an entry, 8-bit states 16): 233 M entries in 1165 us (5.6
// TB/s) and 713 us (5.3 TB/s).  A work-group takes 4096 consecutive entries of
// one tensor, every load of its four steps issued before the first is used.  The
// tensors stand in a table in device memory, where a work-group finds its own by
// comparing 64 tensors' first work-groups at once, one per lane (a level more for
// every 64 times as many).  All tensors of a form are one launch: 140 small ones
// take 4.0 us.
#include <math.h>

#include <type_traits>

#include "common.hpp"
#include "internal.hpp"
#include "policy/internal_policy.hpp"

namespace logra {

namespace {

constexpr int kThreads = 256;
constexpr int kVec = 4;                              // entries per lane and step
constexpr int kStep = kThreads * kVec;               // entries per work-group and step
constexpr int kManySteps = 4;
// Below this many work-groups of kManySteps steps, one step each: 23 ragged tensors
// of 640 k entries with 8-bit states took 11 us in 160 work-groups, 6.1 in steps of
// their own (140 tensors of 1536 and 256 entries the same 4 us, latency).
constexpr int64_t kFew = 1024;

// ---------------------------------------------------------------- 8-bit states
constexpr int kKeepM = 3, kKeepV = 4;            // mantissa bits kept
constexpr int kExpMin = 16, kExpNan = 255;

template <int KEEP>
__device__ __forceinline__ float decode(uint32_t c, int E) {
  const uint32_t b = ((uint32_t)(E - 15) << 23) + (c << (23 - KEEP));
  const float x = c ? __uint_as_float(b) : 0.0f;
  return E == kExpNan ? NAN : x;
}
__device__ __forceinline__ float decode_m(uint32_t code, int E) {
  const float x = decode<kKeepM>(code & 127u, E);
  return (code & 128u) ? -x : x;
}

// Largest value over the eight lanes that hold a block.
__device__ __forceinline__ int block_max(int x) {
  // lanes 1 and 2 apart inside a quad, then the other quad of the half row
  x = max(x, __builtin_amdgcn_mov_dpp(x, 0xB1, 0xF, 0xF, true));    // quad_perm [1,0,3,2]
  x = max(x, __builtin_amdgcn_mov_dpp(x, 0x4E, 0xF, 0xF, true));    // quad_perm [2,3,0,1]
  x = max(x, __builtin_amdgcn_mov_dpp(x, 0x141, 0xF, 0xF, true));   // row_half_mirror
  return x;
}

// Codes of the magnitudes x (>= 0 or NaN) of a lane's entries: packed bytes,
// and the block's exponent.  `least`: a nonzero x keeps a nonzero code.
template <int KEEP>
__device__ __forceinline__ uint32_t encode(const float* x, uint32_t h0, bool least, int* E_out) {
  uint32_t t[kVec];
  int top = 0;
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    // (without a NaN's sign, which the dither would carry out of the word)
    t[e] = __float_as_uint(fabsf(x[e])) + ((h0 + (uint32_t)e * kDitherIndex) >> (9 + KEEP));
    top = max(top, (int)(t[e] >> 23));
  }
  const int E = min(max(block_max(top), kExpMin), kExpNan);
  const int base = (E - 15) << KEEP;
  uint32_t packed = 0;
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    int c = (int)(t[e] >> (23 - KEEP)) - base;
    c = max(c, least && x[e] > 0.0f ? 1 : 0);
    packed |= (uint32_t)min(c, KEEP == kKeepM ? 127 : 255) << (8 * e);
  }
  *E_out = E;
  return packed;
}

// ---------------------------------------------------------------- arrays
// Entries i .. i + 3 of an array (`vec`: one aligned load; else each on its
// own, entries past n not touched).
template <class F>
__device__ __forceinline__ void each(int64_t i, int64_t n, F f) {
#pragma unroll
  for (int e = 0; e < kVec; ++e)
    if (i + e < n) f(e);
}
__device__ __forceinline__ void load4(const float* a, int64_t i, int64_t n, bool vec, float* x) {
  if (vec) {
    const f32x4 q = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(a + i));
#pragma unroll
    for (int e = 0; e < kVec; ++e) x[e] = q[e];
  } else {
    each(i, n, [&](int e) { x[e] = a[i + e]; });
  }
}
__device__ __forceinline__ void load4(const uint16_t* a, int64_t i, int64_t n, bool vec, float* x) {
  if (vec) {
    const u32x2 q = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(a + i));
    x[0] = bf16_lo(q[0]);
    x[1] = bf16_hi(q[0]);
    x[2] = bf16_lo(q[1]);
    x[3] = bf16_hi(q[1]);
  } else {
    each(i, n, [&](int e) { x[e] = bf16_to_f32(a[i + e]); });
  }
}
__device__ __forceinline__ uint32_t load4(const uint8_t* a, int64_t i, int64_t n, bool vec) {
  if (vec) return __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(a + i));
  uint32_t q = 0;
  each(i, n, [&](int e) { q |= (uint32_t)a[i + e] << (8 * e); });
  return q;
}
__device__ __forceinline__ void store4(float* a, int64_t i, int64_t n, bool vec, const float* x) {
  if (vec) {
    const f32x4 q = {x[0], x[1], x[2], x[3]};
    __builtin_nontemporal_store(q, reinterpret_cast<f32x4*>(a + i));
  } else {
    each(i, n, [&](int e) { a[i + e] = x[e]; });
  }
}
__device__ __forceinline__ void store4(uint16_t* a, int64_t i, int64_t n, bool vec,
                                       const float* x) {
  if (vec) {
    const u32x2 q = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
    __builtin_nontemporal_store(q, reinterpret_cast<u32x2*>(a + i));
  } else {
    each(i, n, [&](int e) { a[i + e] = f32_to_bf16(x[e]); });
  }
}
__device__ __forceinline__ void store4(uint8_t* a, int64_t i, int64_t n, bool vec, uint32_t q) {
  if (vec) {
    __builtin_nontemporal_store(q, reinterpret_cast<uint32_t*>(a + i));
  } else {
    each(i, n, [&](int e) { a[i + e] = (uint8_t)(q >> (8 * e)); });
  }
}

// ---------------------------------------------------------------- the step
// Index of the tensor that work-group wg belongs to: the last one whose first
// work-group is not past it.
__device__ __forceinline__ int find_tensor(const int32_t* __restrict__ first, int n, int wg) {
  const int lane = threadIdx.x & 63;
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 63) / 64;
    const int at = lane * step;
    const int before = __popcll(__ballot(at < len && first[lo + (at < len ? at : 0)] <= wg));
    lo += (before - 1) * step;
    len = len - (before - 1) * step < step ? len - (before - 1) * step : step;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

template <AdamwWeights W, bool G32, bool S8, int kSteps>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const AdamwScalars h,
                                                         const AdamwItem* __restrict__ items,
                                                         const int32_t* __restrict__ first,
                                                         int n_items) {
  typedef typename std::conditional<W == AdamwWeights::kF32, float, uint16_t>::type PT;
  typedef typename std::conditional<G32, float, uint16_t>::type GT;
  const int lane = threadIdx.x & 63;
  const int wg = (int)blockIdx.x;
  const int it = find_tensor(first, n_items, wg);
  const AdamwItem& q = items[it];
  PT* const p = static_cast<PT*>(q.p);
  const GT* const g = static_cast<const GT*>(q.g);
  float* const master = q.master;
  void* const mp = q.m;
  void* const vp = q.v;
  uint8_t* const m_exp = q.m_exp;
  uint8_t* const v_exp = q.v_exp;
  const int64_t n = q.n;
  const float wd = q.weight_decay;
  const uint32_t d0 = q.dither0;
  const bool vec_ok = q.vec != 0;
  const float lr = h.lr, b1 = h.b1, b2 = h.b2, c1 = h.c1, c2 = h.c2, eps = h.eps;
  const float ibc1 = h.inv_bc1, isbc2 = h.inv_sqrt_bc2;
  const uint32_t dstep = h.dither_step;
  const float gs = h.grad_scale ? *h.grad_scale : 1.0f;

  const int64_t i0 = (int64_t)(wg - first[it]) * (kStep * kSteps) + (int64_t)threadIdx.x * kVec;
  float xw[kSteps][kVec], xg[kSteps][kVec], xm[kSteps][kVec], xv[kSteps][kVec];
  uint32_t qm[kSteps], qv[kSteps];
  int em[kSteps], ev[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int64_t i = i0 + (int64_t)s * kStep;
    const bool vec = vec_ok && i + kVec <= n;
#pragma unroll
    for (int e = 0; e < kVec; ++e) xw[s][e] = xg[s][e] = xm[s][e] = xv[s][e] = 0.0f;
    qm[s] = qv[s] = 0;
    em[s] = ev[s] = kExpMin;
    if (i < n) {
      if constexpr (W == AdamwWeights::kBf16Master)
        load4(master, i, n, vec, xw[s]);
      else
        load4(p, i, n, vec, xw[s]);
      load4(g, i, n, vec, xg[s]);
      if constexpr (S8) {
        qm[s] = load4(static_cast<const uint8_t*>(mp), i, n, vec);
        qv[s] = load4(static_cast<const uint8_t*>(vp), i, n, vec);
        em[s] = m_exp[i / kStateBlock];
        ev[s] = v_exp[i / kStateBlock];
      } else {
        load4(static_cast<const float*>(mp), i, n, vec, xm[s]);
        load4(static_cast<const float*>(vp), i, n, vec, xv[s]);
      }
    }
  }
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int64_t i = i0 + (int64_t)s * kStep;
    const bool vec = vec_ok && i + kVec <= n;
    float xr[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      if constexpr (S8) {
        xm[s][e] = decode_m((qm[s] >> (8 * e)) & 255u, em[s]);
        const float r = decode<kKeepV>((qv[s] >> (8 * e)) & 255u, ev[s]);
        xv[s][e] = r * r;
      }
      const float gr = xg[s][e] * gs;
      const float m = fmaf(b1, xm[s][e], c1 * gr);
      const float v = fmaf(b2, xv[s][e], c2 * gr * gr);
      const float r = sqrtf(v);
      const float step = (m * ibc1) / fmaf(r, isbc2, eps);
      xw[s][e] = xw[s][e] - lr * fmaf(wd, xw[s][e], step);
      xm[s][e] = m;
      xv[s][e] = v;
      xr[e] = r;
    }
    if constexpr (S8) {
      // (entries past n are zeros here; every lane takes part in the block's
      // maximum)
      const uint32_t h = (d0 + (uint32_t)i) * kDitherIndex + dstep;
      float xa[kVec];
      uint32_t sign = 0;
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        xa[e] = fabsf(xm[s][e]);
        sign |= (__float_as_uint(xm[s][e]) >> 31) << (8 * e + 7);
        if (i + e >= n) xa[e] = xr[e] = 0.0f;
      }
      int E;
      const uint32_t cm = encode<kKeepM>(xa, h, false, &E) | sign;
      em[s] = E;
      const uint32_t cv = encode<kKeepV>(xr, h + 0x80000000u, true, &E);
      ev[s] = E;
      qm[s] = cm;
      qv[s] = cv;
    }
    if (i < n) {
      store4(p, i, n, vec, xw[s]);
      if constexpr (W == AdamwWeights::kBf16Master) store4(master, i, n, vec, xw[s]);
      if constexpr (S8) {
        store4(static_cast<uint8_t*>(mp), i, n, vec, qm[s]);
        store4(static_cast<uint8_t*>(vp), i, n, vec, qv[s]);
        if ((lane & 7) == 0) {
          m_exp[i / kStateBlock] = (uint8_t)em[s];
          v_exp[i / kStateBlock] = (uint8_t)ev[s];
        }
      } else {
        store4(static_cast<float*>(mp), i, n, vec, xm[s]);
        store4(static_cast<float*>(vp), i, n, vec, xv[s]);
      }
    }
  }
}

// Two values as bf16 in one word, from codes in the low bytes of its halves: every
// value of the form is exact in bf16, so both are formed at once by integer
// arithmetic that does not cross the halves.  base: (E - 15) << 7 in each.
template <bool SECOND>
__device__ __forceinline__ uint32_t value_pair(uint32_t w, uint32_t base) {
  const uint32_t c = SECOND ? w : w & 0x007F007Fu;
  const uint32_t t = (c + 0x00FF00FFu) & 0x01000100u;        // where c is not 0
  uint32_t x = (base + (c << (7 - (SECOND ? kKeepV : kKeepM)))) & ((t << 8) - (t >> 8));
  if constexpr (!SECOND) x |= (w & 0x00800080u) << 8;
  return x;
}

// Eight entries per lane and step, four steps: 8-byte loads and 16-byte stores that
// cover whole lines in every instruction (with 16 entries a lane, each store had
// every other 16 bytes of its lines, 181 and 132 us).  233 M entries: 116 us, 6.2
// TB/s.
constexpr int kValues = 8;
constexpr int kValueSteps = 4;

template <bool SECOND>
__global__ __launch_bounds__(kThreads) void state_values_kernel(const uint8_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ exps,
                                                                int64_t n, bool vec_ok,
                                                                uint16_t* __restrict__ out) {
  constexpr int64_t kCols = kThreads * kValues;
  for (int64_t i0 = (int64_t)blockIdx.x * (kCols * kValueSteps); i0 < n;
       i0 += (int64_t)gridDim.x * (kCols * kValueSteps)) {
    const int64_t i = i0 + (int64_t)threadIdx.x * kValues;
    u32x2 q[kValueSteps];
    uint32_t E[kValueSteps];
#pragma unroll
    for (int s = 0; s < kValueSteps; ++s) {
      const int64_t at = i + s * kCols;
      q[s] = u32x2{0, 0};
      E[s] = kExpMin;
      if (at < n) E[s] = exps[at / kStateBlock];
      if (vec_ok && at + kValues <= n)
        q[s] = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(codes + at));
    }
#pragma unroll
    for (int s = 0; s < kValueSteps; ++s) {
      const int64_t at = i + s * kCols;
      if (vec_ok && at + kValues <= n) {
        const uint32_t base = ((E[s] - 15) << 7) * 0x10001u;
        const uint32_t nan = E[s] == kExpNan ? 0x7FC07FC0u : 0;
        u32x4 v;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t w =
              __builtin_amdgcn_perm(0, q[s][p >> 1], (p & 1) ? 0x0C030C02u : 0x0C010C00u);
          v[p] = value_pair<SECOND>(w, base) | nan;
        }
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(out + at));
      } else {
        for (int e = 0; e < kValues && at + e < n; ++e) {
          const uint32_t c = codes[at + e];
          out[at + e] = f32_to_bf16(SECOND ? decode<kKeepV>(c, (int)E[s]) : decode_m(c, (int)E[s]));
        }
      }
    }
  }
}

bool on(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <AdamwWeights W, bool G32, bool S8>
void launch_form(int steps, int64_t groups, const AdamwScalars& h, const AdamwItem* items,
                 const int32_t* first, int n, hipStream_t s) {
  const dim3 grid((unsigned)groups), block(kThreads);
  if (steps == 1)
    hipLaunchKernelGGL((adamw_kernel<W, G32, S8, 1>), grid, block, 0, s, h, items, first, n);
  else
    hipLaunchKernelGGL((adamw_kernel<W, G32, S8, kManySteps>), grid, block, 0, s, h, items, first,
                       n);
}

template <AdamwWeights W>
void launch_weights(bool g_f32, bool state8, int steps, int64_t groups, const AdamwScalars& h,
                    const AdamwItem* items, const int32_t* first, int n, hipStream_t s) {
  if (g_f32) {
    if (state8)
      launch_form<W, true, true>(steps, groups, h, items, first, n, s);
    else
      launch_form<W, true, false>(steps, groups, h, items, first, n, s);
  } else {
    if (state8)
      launch_form<W, false, true>(steps, groups, h, items, first, n, s);
    else
      launch_form<W, false, false>(steps, groups, h, items, first, n, s);
  }
}

}  // namespace

bool adamw_lay_out(AdamwForm* form, AdamwItem* items, int32_t* first, bool g_f32, bool state8,
                   AdamwWeights weights) {
  int64_t groups = 0;
  for (int i = 0; i < form->n; ++i) groups += (items[i].n + kStep * kManySteps - 1) / (kStep * kManySteps);
  form->steps = groups < kFew ? 1 : kManySteps;
  const int64_t chunk = (int64_t)kStep * form->steps;
  const uintptr_t pb = weights == AdamwWeights::kF32 ? 4 : 2, gb = g_f32 ? 4 : 2;
  const uintptr_t sb = state8 ? 1 : 4;
  groups = 0;
  for (int i = 0; i < form->n; ++i) {
    AdamwItem& q = items[i];
    q.vec = on(q.p, kVec * pb) && on(q.g, kVec * gb) && on(q.master, kVec * 4) &&
            on(q.m, kVec * sb) && on(q.v, kVec * sb);
    first[i] = (int32_t)groups;
    groups += (q.n + chunk - 1) / chunk;
    if (groups >= (int64_t(1) << 24)) return false;   // 2^32 threads
  }
  form->groups = (int32_t)groups;
  return true;
}

hipError_t launch_adamw(AdamwWeights weights, bool g_f32, bool state8, const AdamwForm& form,
                        const AdamwItem* items, const int32_t* first, const AdamwScalars& h,
                        hipStream_t s) {
  switch (weights) {
    case AdamwWeights::kF32:
      launch_weights<AdamwWeights::kF32>(g_f32, state8, form.steps, form.groups, h, items, first,
                                         form.n, s);
      break;
    case AdamwWeights::kBf16:
      launch_weights<AdamwWeights::kBf16>(g_f32, state8, form.steps, form.groups, h, items, first,
                                          form.n, s);
      break;
    default:
      launch_weights<AdamwWeights::kBf16Master>(g_f32, state8, form.steps, form.groups, h, items,
                                                first, form.n, s);
  }
  return hipGetLastError();
}

hipError_t launch_adamw_state_values(bool second, const uint8_t* codes, const uint8_t* exps,
                                     int64_t n, uint16_t* out, hipStream_t s) {
  int64_t blocks = (n + kThreads * kValues * kValueSteps - 1) / (kThreads * kValues * kValueSteps);
  if (blocks > (1 << 20)) blocks = 1 << 20;
  const bool vec = on(codes, 8) && on(out, 16);
  if (second)
    hipLaunchKernelGGL((state_values_kernel<true>), dim3((unsigned)blocks), dim3(kThreads), 0, s,
                       codes, exps, n, vec, out);
  else
    hipLaunchKernelGGL((state_values_kernel<false>), dim3((unsigned)blocks), dim3(kThreads), 0, s,
                       codes, exps, n, vec, out);
  return hipGetLastError();
}

}  // namespace logra
