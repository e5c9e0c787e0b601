// logra_adapter_apply: out[t] = RNE_bf16(Y[t] + c scale[a] (X[t] A_a^T) U_a^T),
// a = adapter[t], on gfx950: the rank-r updates of several policies beside the
// projection they share.
//
// [LoGRA] (wispaper.ai summary of "LoGRA: Scaling LLM Reinforcement Learning
// with Low-Rank Gradient Sketches"), sections Sketch and Sync: a layer's update
// is W - alpha eta U A with A rebuilt from a seed; here it meets the layer's
// input instead of its weights.
//
// Two launches:
//   project  P = X A^T, fp32, for 32 rows and a piece of k per work-group.  The
//            rank is the MFMA's row index and the tokens its columns, so a
//            token's values lie in the lanes of its own column and the rows of
//            a tile that belong to other policies (or hold NaN) touch nothing.
//            A tile's policies are found by ballots and taken one after the
//            other, or dealt to several work-groups where few tiles leave the
//            chip empty; each writes the P of its own rows.  Signs: one Philox
//            block per thread gives 256 rows x 256 columns' worth at a time
//            (rows x chunks), kept in LDS and expanded to +-1 in registers, so
//            a seeded A is never read: a decoding batch over many policies
//            streams only U.
//   expand   out = Y + P U^T for 64 rows (16 for few rows) x 64 columns per
//            wave.  U's rows are the MFMA's rows, in the order that leaves each
//            lane 16 consecutive columns of one token.  P (its pieces summed in
//            order and scaled) and fp32 U enter as bf16 pairs hi + lo of 16
//            significant bits; lo x lo, 2^-16 of the product, is left out.  The
//            rows of each policy are written as soon as it is done; rows with
//            none are copied.
// Bound: X and Y once in, out once (prompts); U of every policy in use, and
// launch latency (single tokens).
#include "common.hpp"
#include "internal.hpp"
#include "policy/internal_policy.hpp"

namespace logra {

namespace {

constexpr int kThreads = 256;
constexpr int kTileRows = 32;      // rows of a projection tile
constexpr int kChunk = 256;        // columns of a sign block

// ---------------------------------------------------------------- the policies of a tile
// Lane l holds row l's policy (-1: none).  next() gives the policies in the
// order of their first rows.
struct Policies {
  int id;
  uint64_t left;
  __device__ __forceinline__ Policies(const int32_t* adapter, int64_t row, bool in, int64_t n) {
    id = in ? adapter[row] : -1;
    if (id < 0 || (int64_t)id >= n) id = -1;
    left = __ballot(id >= 0);
  }
  __device__ __forceinline__ bool next(int* a, uint64_t* rows) {
    if (left == 0) return false;
    *a = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)left) - 1);
    *rows = __ballot(id == *a);
    left &= ~*rows;
    return true;
  }
};

// Elements col .. col + 7 of a bf16 row of n, those past n as zeros (and not
// read: the last row of a matrix need not have padding behind it).
__device__ __forceinline__ u32x4 load_row8(const uint16_t* row, int col, int n) {
  if (col + 8 <= n) return load_bf16x8(row, col);
  u32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (col + e < n) v[e >> 1] |= (uint32_t)row[col + e] << (16 * (e & 1));
  return v;
}

// ---------------------------------------------------------------- project
// NB 16-row blocks of A: per wave kNbw of them, kKsub waves sharing a block and
// splitting its steps of 32 columns.
template <int NB, bool GIVEN>
__global__ __launch_bounds__(kThreads) void adapter_project_kernel(AdapterArgs a, int n_split,
                                                                   int chunks_per_split, int n_deal,
                                                                   float* __restrict__ P) {
  constexpr int RP = 16 * NB;
  constexpr int kGroups = NB < 4 ? NB : 4;
  constexpr int kKsub = 4 / kGroups;
  constexpr int kNbw = NB / kGroups;
  constexpr int kSuper = 256 / RP;          // chunks whose signs fit one pass
  constexpr int kRowBytes = kChunk * 2;
  __shared__ __attribute__((aligned(16))) unsigned char xs[kTileRows * kRowBytes];
  __shared__ uint64_t sgn[GIVEN ? 1 : 256 * 4];
  __shared__ f32x4 red[kKsub > 1 ? 4 * 2 * kNbw * 64 : 1];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = tid >> 6;
  const int m = lane & 15;    // row of A in its block; token in its block
  const int g = lane >> 4;    // 64-column quarter of a chunk
  const int grp = wave / kKsub, ksub = wave % kKsub;
  const SignMasks smk = sign_masks();

  const int n_tiles = (int)((a.T + kTileRows - 1) / kTileRows);
  const int tile = (int)(blockIdx.x % n_tiles);
  const int rest = (int)(blockIdx.x / n_tiles);
  const int split = rest % n_split;
  const int deal = rest / n_split;
  const int64_t t0 = (int64_t)tile * kTileRows;
  const int n_chunks = (a.k + kChunk - 1) / kChunk;
  const int ch0 = split * chunks_per_split;
  const int ch1 = ch0 + chunks_per_split < n_chunks ? ch0 + chunks_per_split : n_chunks;

  Policies pol(a.adapter, t0 + lane, lane < kTileRows && t0 + lane < a.T, a.n);
  int id;
  uint64_t rows;
  for (int u = 0; pol.next(&id, &rows); ++u) {
    if (u % n_deal != deal) continue;
    uint64_t seed = 0, stream = 0;
    const uint16_t* A = nullptr;
    if constexpr (GIVEN) {
      A = a.A + (int64_t)id * a.r * a.lda;
    } else {
      seed = a.seeds[2 * (int64_t)id];
      stream = a.seeds[2 * (int64_t)id + 1];
    }
    f32x4 acc[kNbw][2];
#pragma unroll
    for (int b = 0; b < kNbw; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h) acc[b][h] = f32x4{0.f, 0.f, 0.f, 0.f};

    // this thread's four 16-byte pieces of a chunk's X tile
    u32x4 xr[4];
    auto fetch = [&](int ch) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t t = t0 + (tid >> 5) + 8 * i;
        const uint16_t* row = a.X + (t < a.T ? t : a.T - 1) * a.ldx;
        xr[i] = load_row8(row, ch * kChunk + 8 * (tid & 31), a.k);
      }
    };
    if (ch0 < ch1) fetch(ch0);
    for (int ch = ch0; ch < ch1; ++ch) {
      __syncthreads();   // xs, sgn and red are free
      if constexpr (!GIVEN) {
        const int sc = (ch - ch0) % kSuper;
        if (sc == 0) {
          const int c = ch + tid / RP;
          if (c < ch1) {
            const Words4 w = sign_block(seed, stream, (uint64_t)c, (uint64_t)(tid % RP));
#pragma unroll
            for (int q = 0; q < 4; ++q) sgn[tid * 4 + q] = w.w[q];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = (tid >> 5) + 8 * i, j = tid & 31;
        const int slot = (j & 16) | ((j ^ row) & 15);
        *reinterpret_cast<u32x4*>(xs + row * kRowBytes + slot * 16) = xr[i];
      }
      __syncthreads();
      if (ch + 1 < ch1) fetch(ch + 1);
      uint64_t sw[kNbw];
      if constexpr (!GIVEN) {
#pragma unroll
        for (int b = 0; b < kNbw; ++b)
          sw[b] = sgn[(((ch - ch0) % kSuper) * RP + (grp * kNbw + b) * 16 + m) * 4 + g];
      }
#pragma unroll
      for (int ss = 0; ss < 8 / kKsub; ++ss) {
        const int s = ss * kKsub + ksub;
        const int j = 8 * g + s;
        u32x4 x[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = 16 * h + m;
          const int slot = (j & 16) | ((j ^ row) & 15);
          x[h] = *reinterpret_cast<const u32x4*>(xs + row * kRowBytes + slot * 16);
        }
#pragma unroll
        for (int b = 0; b < kNbw; ++b) {
          u32x4 w;
          if constexpr (GIVEN) {
            const int i = (grp * kNbw + b) * 16 + m;
            w = load_row8(A + (int64_t)(i < a.r ? i : a.r - 1) * a.lda, ch * kChunk + 8 * j, a.k);
          } else {
            w = signs_to_bf16x8((uint32_t)(sw[b] >> (8 * s)) & 0xFFu, smk);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) acc[b][h] = mfma16(w, x[h], acc[b][h]);
        }
      }
    }
    if constexpr (kKsub > 1) {
      // the waves of a block meet in LDS, in order
      __syncthreads();
#pragma unroll
      for (int b = 0; b < kNbw; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) red[((wave * kNbw + b) * 2 + h) * 64 + lane] = acc[b][h];
      __syncthreads();
      if (ksub == 0) {
#pragma unroll
        for (int b = 0; b < kNbw; ++b)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int q = 1; q < kKsub; ++q)
              acc[b][h] += red[(((wave + q) * kNbw + b) * 2 + h) * 64 + lane];
      }
    }
    if (ksub == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 16 * h + m;
        if ((rows >> row) & 1) {
          float* p = P + ((int64_t)split * a.T + t0 + row) * RP;
#pragma unroll
          for (int b = 0; b < kNbw; ++b) {
            const int i = (grp * kNbw + b) * 16 + 4 * g;
            f32x4 v = acc[b][h];
            // columns past r meet no U
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = i + e < a.r ? v[e] : 0.0f;
            *reinterpret_cast<f32x4*>(p + i) = v;
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------- expand
__device__ __forceinline__ void split8(const float* x, u32x4& hi, u32x4& lo) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    hi[p] = pack_bf16x2(x[2 * p], x[2 * p + 1]);
    lo[p] = pack_bf16x2(x[2 * p] - bf16_lo(hi[p]), x[2 * p + 1] - bf16_hi(hi[p]));
  }
}

// Elements K .. K + 7 of a row of U (r of them), those past r as zeros.
template <bool VEC>
__device__ __forceinline__ void load_u(const float* row, int K, int r, u32x4& hi, u32x4& lo) {
  float x[8];
  if (VEC) {
    const int at = K < r ? K : 0;
    const f32x4 u = *reinterpret_cast<const f32x4*>(row + at);
    const f32x4 v = *reinterpret_cast<const f32x4*>(row + at + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = K < r ? u[e] : 0.0f;
      x[4 + e] = K < r ? v[e] : 0.0f;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = K + e < r ? row[K + e] : 0.0f;
  }
  split8(x, hi, lo);
}
template <bool VEC>
__device__ __forceinline__ void load_u(const uint16_t* row, int K, int r, u32x4& hi, u32x4& lo) {
  if (VEC) {
    hi = load_bf16x8_masked(row, K, r);
  } else {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t x0 = K + 2 * p < r ? row[K + 2 * p] : 0;
      const uint32_t x1 = K + 2 * p + 1 < r ? row[K + 2 * p + 1] : 0;
      hi[p] = x0 | (x1 << 16);
    }
  }
  lo = u32x4{0, 0, 0, 0};
}

// 8 columns of one row of out = Y + delta (or the bits of Y, COPY).
template <bool COPY>
__device__ __forceinline__ void write8(const uint16_t* y, uint16_t* o, int col, int d,
                                       const float* delta) {
  if (col + 8 <= d) {
    u32x4 v = *reinterpret_cast<const u32x4*>(y + col);
    if constexpr (!COPY) {
#pragma unroll
      for (int p = 0; p < 4; ++p)
        v[p] = pack_bf16x2(bf16_lo(v[p]) + delta[2 * p], bf16_hi(v[p]) + delta[2 * p + 1]);
    }
    *reinterpret_cast<u32x4*>(o + col) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + e < d) {
        if constexpr (COPY)
          o[col + e] = y[col + e];
        else
          o[col + e] = f32_to_bf16(bf16_to_f32(y[col + e]) + delta[e]);
      }
  }
}

// NR blocks of 16 rows x 64 columns per wave, NW waves side by side along d.
// RP: row length of P; NKS steps of 32 along the rank.
template <int RP, class UT, bool VEC, int NR, int NW>
__global__ __launch_bounds__(64 * NW) void adapter_expand_kernel(AdapterArgs a, int n_split,
                                                                 float c, const float* __restrict__ P) {
  constexpr int NKS = RP < 32 ? 1 : RP / 32;
  constexpr bool kPair = sizeof(UT) == 4;   // U as hi + lo
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int m = lane & 15;
  const int g = lane >> 4;
  const int n_cb = (a.d + 64 * NW - 1) / (64 * NW);
  const int64_t rb0 = (int64_t)(blockIdx.x / n_cb) * (16 * NR);
  const int col0 = ((int)(blockIdx.x % n_cb) * NW + wave) * 64;
  if (col0 >= a.d) return;
  const int64_t myrow = rb0 + lane;
  Policies pol(a.adapter, myrow, lane < 16 * NR && myrow < a.T, a.n);

  // rows without a policy
  if (a.out != a.Y) {
    const uint64_t none = __ballot(lane < 16 * NR && myrow < a.T) & ~pol.left;
    if (none) {
#pragma unroll
      for (int b = 0; b < NR; ++b) {
        const int64_t t = rb0 + 16 * b + m;
        if ((none >> (16 * b + m)) & 1) {
          write8<true>(a.Y + t * a.ldy, a.out + t * a.ldo, col0 + 16 * g, a.d, nullptr);
          write8<true>(a.Y + t * a.ldy, a.out + t * a.ldo, col0 + 16 * g + 8, a.d, nullptr);
        }
      }
    }
  }

  int id;
  uint64_t rows;
  while (pol.next(&id, &rows)) {
    const UT* U = static_cast<const UT*>(a.U) + (int64_t)id * a.d * a.r;
    const float sc = c * a.scale[id];
    f32x4 acc[NR][4];
#pragma unroll
    for (int b = 0; b < NR; ++b)
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[b][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int s = 0; s < NKS; ++s) {
      const int K = 32 * s + 8 * g;
      u32x4 uh[4], ul[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int col = col0 + (m >> 2) * 16 + 4 * t + (m & 3);
        load_u<VEC>(U + (int64_t)(col < a.d ? col : a.d - 1) * a.r, K, a.r, uh[t], ul[t]);
      }
#pragma unroll
      for (int b = 0; b < NR; ++b) {
        if (((rows >> (16 * b)) & 0xFFFFu) == 0) continue;
        // rows of other policies give columns that are not used
        const int64_t row = rb0 + 16 * b + m;
        const int64_t t = row < a.T ? row : a.T - 1;
        float p[8] = {};
        if (RP >= 32 || K < RP) {
          for (int q = 0; q < n_split; ++q) {
            const float* src = P + ((int64_t)q * a.T + t) * RP + K;
            const f32x4 lo4 = *reinterpret_cast<const f32x4*>(src);
            const f32x4 hi4 = *reinterpret_cast<const f32x4*>(src + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              p[e] += lo4[e];
              p[4 + e] += hi4[e];
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] *= sc;
        u32x4 ph, pl;
        split8(p, ph, pl);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          acc[b][w] = mfma16(uh[w], pl, acc[b][w]);
          if constexpr (kPair) acc[b][w] = mfma16(ul[w], ph, acc[b][w]);
          acc[b][w] = mfma16(uh[w], ph, acc[b][w]);
        }
      }
    }
#pragma unroll
    for (int b = 0; b < NR; ++b) {
      if ((rows >> (16 * b + m)) & 1) {
        const int64_t t = rb0 + 16 * b + m;
        float delta[16];
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int e = 0; e < 4; ++e) delta[4 * w + e] = acc[b][w][e];
        write8<false>(a.Y + t * a.ldy, a.out + t * a.ldo, col0 + 16 * g, a.d, delta);
        write8<false>(a.Y + t * a.ldy, a.out + t * a.ldo, col0 + 16 * g + 8, a.d, delta + 8);
      }
    }
  }
}

// ---------------------------------------------------------------- launches
constexpr int64_t kFill = 512;   // work-groups that keep the chip busy

template <int NB>
void launch_project(const AdapterArgs& a, const AdapterPlan& p, float* P, hipStream_t s) {
  const int64_t tiles = (a.T + kTileRows - 1) / kTileRows;
  const int64_t base = tiles * p.n_split;
  int64_t deal = (kFill + base - 1) / base;
  if (deal > kTileRows) deal = kTileRows;
  if (deal > a.n) deal = a.n;
  const dim3 grid((unsigned)(base * deal));
  if (a.A)
    hipLaunchKernelGGL((adapter_project_kernel<NB, true>), grid, dim3(kThreads), 0, s, a, p.n_split,
                       p.chunks_per_split, (int)deal, P);
  else
    hipLaunchKernelGGL((adapter_project_kernel<NB, false>), grid, dim3(kThreads), 0, s, a,
                       p.n_split, p.chunks_per_split, (int)deal, P);
}

template <int RP, class UT, bool VEC>
void launch_expand_vec(const AdapterArgs& a, const AdapterPlan& p, float c, const float* P,
                       hipStream_t s) {
  const int64_t big = ((a.T + 63) / 64) * ((a.d + 255) / 256);
  if (big >= kFill / 2) {
    hipLaunchKernelGGL((adapter_expand_kernel<RP, UT, VEC, 4, 4>), dim3((unsigned)big), dim3(256), 0,
                       s, a, p.n_split, c, P);
  } else {
    const int64_t small = ((a.T + 15) / 16) * ((a.d + 63) / 64);
    hipLaunchKernelGGL((adapter_expand_kernel<RP, UT, VEC, 1, 1>), dim3((unsigned)small), dim3(64),
                       0, s, a, p.n_split, c, P);
  }
}

template <int RP>
void launch_both(const AdapterArgs& a, bool u_f32, const AdapterPlan& p, float c, float* P,
                 hipStream_t s) {
  launch_project<RP / 16>(a, p, P, s);
  const bool vec = a.r % 8 == 0 && (reinterpret_cast<uintptr_t>(a.U) & 15) == 0;
  if (u_f32) {
    if (vec)
      launch_expand_vec<RP, float, true>(a, p, c, P, s);
    else
      launch_expand_vec<RP, float, false>(a, p, c, P, s);
  } else {
    if (vec)
      launch_expand_vec<RP, uint16_t, true>(a, p, c, P, s);
    else
      launch_expand_vec<RP, uint16_t, false>(a, p, c, P, s);
  }
}

}  // namespace

bool make_adapter_plan(int64_t T, int64_t d, int64_t k, int r, AdapterPlan* p) {
  constexpr int64_t kDim = int64_t(1) << 31;
  if (T < 1 || d < 1 || k < 1 || T >= kDim || d >= kDim || k >= kDim || r < 1 || r > 256)
    return false;
  p->rp = r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : r <= 128 ? 128 : 256;
  const int64_t tiles = (T + kTileRows - 1) / kTileRows;
  const int64_t chunks = (k + kChunk - 1) / kChunk;
  int64_t split = (kFill + tiles - 1) / tiles;
  if (split > chunks) split = chunks;
  if (split > 16) split = 16;
  const int64_t per = (chunks + split - 1) / split;
  p->chunks_per_split = (int)per;
  p->n_split = (int)((chunks + per - 1) / per);
  p->total = (size_t)round_up((int64_t)p->n_split * T * p->rp * 4, 256);
  // (flat grids: work-groups, and threads below 2^32)
  const int64_t most = (int64_t(1) << 24) - 1;
  return tiles * p->n_split <= most && ((T + 63) / 64) * ((d + 255) / 256) <= most;
}

hipError_t launch_adapter(const AdapterArgs& a, bool u_f32, const AdapterPlan& p, char* ws,
                          hipStream_t s) {
  float* P = reinterpret_cast<float*>(ws);
  const float c = a.A ? 1.0f : sign_scale(a.r);
  switch (p.rp) {
    case 16: launch_both<16>(a, u_f32, p, c, P, s); break;
    case 32: launch_both<32>(a, u_f32, p, c, P, s); break;
    case 64: launch_both<64>(a, u_f32, p, c, P, s); break;
    case 128: launch_both<128>(a, u_f32, p, c, P, s); break;
    default: launch_both<256>(a, u_f32, p, c, P, s); break;
  }
  return hipGetLastError();
}

}  // namespace logra
