// logra_linear and its gradients: a layer's product with bias, activation and
// residual in its epilogue, and the products of its backward pass, on gfx950.
//
// All three products are C(m, n) = sum over K of A(m, k) B(n, k) in bf16 with fp32
// sums on the matrix cores; they differ in which way their operands lie:
//   forward   X [T, k] W [d, k]^T   both with K contiguous
//   input     dY [T, d] W [d, k]    W has K along its rows
//   weight    dY [T, d]^T X [T, k]  both have K (= T) along their rows
// An operand with K contiguous is read from LDS 16 bytes a lane, as a 16x16x32
// operand takes it; one with K along its rows through the transposing LDS read (four
// rows by 16 columns per 16 lanes).  Either way lane group g holds K indices 8 g ..
// 8 g + 7 of 32, so the two kinds meet in any combination.
//
// Bound: the matrix cores' power for large products (the clock falls to 1.5 - 1.9 GHz
// under them; a loop of nothing but 32x32x16 products of random numbers reaches 1830
// TFLOP/s, 16x16x32 ones 1700): 8192 x 4096 x 4096 takes 218, 210 and 209 us in the three
// forms (1260 to 1315 TFLOP/s; the library's products 179, 212 and 232); the weights' HBM
// bytes for few rows (64 x 1536 to 152064 fp32 results: 98 us, 5.2 TB/s).
#include <math.h>

#include "common.hpp"
#include "internal.hpp"
#include "step/internal_step.hpp"

namespace logra {

namespace {

constexpr int kBK = 64;         // K of one step

typedef short s16x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ activations
__device__ __forceinline__ float rcp(float x) { return __builtin_amdgcn_rcpf(x); }
// 1 / (1 + e^-x)
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + __expf(-x)); }

// Phi(-|x|) and e^(-x^2 / 2) of the normal distribution.  Phi(-z) e^(z^2 / 2) is t
// times a polynomial of degree 7 in t = 1 / (1 + 0.3 z), fitted over z in [0, 14] to
// the least largest relative error (1.5e-7; 5e-7 in fp32 arithmetic), so that the far
// side keeps its digits: erfcf's branches cost five times as much and took 80 us of
// a product of 8192 x 4096 results.
__device__ __forceinline__ float tail(float x, float* e) {
  const float t = rcp(fmaf(0.3f, fabsf(x), 1.f));
  *e = __expf(-0.5f * x * x);
  float p = 0x1.243fb4p-5f;
  p = fmaf(p, t, -0x1.41f3f6p-3f);
  p = fmaf(p, t, 0x1.a69d18p-3f);
  p = fmaf(p, t, -0x1.b7c826p-5f);
  p = fmaf(p, t, 0x1.074b7ap-3f);
  p = fmaf(p, t, 0x1.993ecep-4f);
  p = fmaf(p, t, 0x1.ee9bb6p-4f);
  p = fmaf(p, t, 0x1.ea006ap-4f);
  return p * t * *e;
}

constexpr float kGeluA = 1.5957691216057308f;    // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

template <int ACT>
__device__ __forceinline__ float activate(float x) {
  if constexpr (ACT == kActRelu) return x > 0.f || x != x ? x : 0.f;
  if constexpr (ACT == kActSilu) return x * sigmoid(x);
  if constexpr (ACT == kActGelu) {
    float e;
    const float q = tail(x, &e);
    // (from 100 on q is 0: clamped there, +inf is not inf times 0)
    return fmaf(x > 0.f ? -fminf(x, 100.f) : x, q, x > 0.f || x != x ? x : 0.f);
  }
  if constexpr (ACT == kActGeluTanh) return x * sigmoid(kGeluA * fmaf(kGeluB * x * x, x, x));
  return x;
}
template <int ACT>
__device__ __forceinline__ float slope(float x) {
  // (from 100 on the slope is 0 or 1 in fp32, and no product below is inf times 0)
  if (fabsf(x) > 100.f) x = copysignf(100.f, x);
  if constexpr (ACT == kActRelu) return x > 0.f ? 1.f : x != x ? x : 0.f;
  if constexpr (ACT == kActSilu) return sigmoid(x) * fmaf(x, sigmoid(-x), 1.f);
  if constexpr (ACT == kActGelu) {
    float e;
    const float q = tail(x, &e);
    return fmaf(x * 0.39894228040143268f, e, x > 0.f ? 1.f - q : q);
  }
  if constexpr (ACT == kActGeluTanh) {
    const float y = kGeluA * fmaf(kGeluB * x * x, x, x);
    const float dy = kGeluA * fmaf(3.f * kGeluB, x * x, 1.f);
    return sigmoid(y) * fmaf(x * dy, sigmoid(-y), 1.f);
  }
  return 1.f;
}
__device__ __forceinline__ float activate_any(float x, int act) {
  switch (act) {
    case kActRelu: return activate<kActRelu>(x);
    case kActSilu: return activate<kActSilu>(x);
    case kActGelu: return activate<kActGelu>(x);
    case kActGeluTanh: return activate<kActGeluTanh>(x);
    default: return x;
  }
}

// ------------------------------------------------------------------ epilogue
__device__ __forceinline__ u32x4 pack8(const float* v) {
  return u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
               pack_bf16x2(v[6], v[7])};
}
// The bias of columns n .. n + 7 (zeros without one, and past the end).
__device__ __forceinline__ void load_bias(const GemmArgs& g, int n, float* b) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    b[e] = 0.f;
    if (g.bias != nullptr && n + e < g.N)
      b[e] = g.bias_f32 ? static_cast<const float*>(g.bias)[n + e]
                        : bf16_to_f32(static_cast<const uint16_t*>(g.bias)[n + e]);
  }
}
// The residual there (zeros without one, and outside the result).
__device__ __forceinline__ u32x4 load_residual(const GemmArgs& g, int m, int n) {
  u32x4 q{0, 0, 0, 0};
  if (g.add != nullptr && m < g.M && n < g.N)
    q = *reinterpret_cast<const u32x4*>(g.add + (int64_t)m * g.ldadd + n);
  return q;
}
// Columns n .. n + 7 of row m (n a multiple of 8, below N), from the sums v and the
// residual q.
__device__ __forceinline__ void epilogue8(const GemmArgs& g, int m, int n, const float* bias,
                                          u32x4 q, float* v) {
  const int valid = g.N - n;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] += bias[e];
  if (g.pre != nullptr) {
    uint16_t* const p = g.pre + (int64_t)m * g.ldpre + n;
    if (valid >= 8) {
      *reinterpret_cast<u32x4*>(p) = pack8(v);
    } else {
      for (int e = 0; e < valid; ++e) p[e] = f32_to_bf16(v[e]);
    }
  }
  if (g.act != kActNone) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = activate_any(v[e], g.act);
  }
  if (g.add != nullptr) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] += bf16_lo(q[e]);
      v[2 * e + 1] += bf16_hi(q[e]);
    }
  }
  if (g.c_f32) {
    float* const p = static_cast<float*>(g.C) + (int64_t)m * g.ldc + n;
    if (valid >= 8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f32x4* const q = reinterpret_cast<f32x4*>(p) + h;
        const f32x4 x{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
        *q = g.accumulate ? *q + x : x;
      }
    } else {
      for (int e = 0; e < valid; ++e) p[e] = g.accumulate ? p[e] + v[e] : v[e];
    }
  } else {
    uint16_t* const p = static_cast<uint16_t*>(g.C) + (int64_t)m * g.ldc + n;
    if (valid >= 8) {
      *reinterpret_cast<u32x4*>(p) = pack8(v);
    } else {
      for (int e = 0; e < valid; ++e) p[e] = f32_to_bf16(v[e]);
    }
  }
}

// ------------------------------------------------------------------ operand tiles in LDS
// R rows (m or n) by kBK, 16-byte pieces.  K contiguous: R rows of 128 bytes, piece c
// of row r at place c ^ (r & 7).  Along K: kBK rows of 2 R bytes, piece c of row k at
// place c ^ 2 (k & 3), so that the four rows a transposing read takes lie in
// different banks.
template <int R, int NW, bool ALONG>
struct Operand {
  static constexpr int kBytes = R * kBK * 2;
  static constexpr int kDma = kBytes / 1024 / NW;        // copies of a wave per step
  static constexpr int kRowPieces = ALONG ? R / 8 : 8;   // 16-byte pieces of an LDS row
  static_assert(kDma * NW * 1024 == kBytes, "whole copies");
  const uint16_t* src[kDma];     // this lane's source in step 0
  int64_t advance;               // elements from one step to the next

  // LDS row and source piece of this lane in copy i.
  __device__ __forceinline__ static void at(int wave, int lane, int i, int* row, int* piece) {
    const int q = (wave * kDma + i) * 64 + lane;
    *row = q / kRowPieces;
    *piece = (q % kRowPieces) ^ (ALONG ? 2 * (*row & 3) : *row & 7);
  }
  // base: the operand; r0: the tile's first row (m or n) of `rows`; k0: first K
  __device__ __forceinline__ void init(const uint16_t* base, int64_t ld, int r0, int rows, int k0,
                                       int wave, int lane) {
    advance = ALONG ? ld * kBK : kBK;
#pragma unroll
    for (int i = 0; i < kDma; ++i) {
      int row, piece;
      at(wave, lane, i, &row, &piece);
      if (ALONG) {
        // (columns past the matrix read its last piece; they reach no stored result)
        const int last = (rows + 7) / 8 * 8 - 8;
        const int col = r0 + piece * 8;
        src[i] = base + (int64_t)(k0 + row) * ld + (col < last ? col : last);
      } else {
        const int r = r0 + row < rows ? r0 + row : rows - 1;
        src[i] = base + (int64_t)r * ld + k0 + piece * 8;
      }
    }
  }
  // Copies [i0, i1) of this lane's next step; a step's copies are issued once each.
  // ONCE: of an operand that no other work-group reads.
  template <bool ONCE = false>
  __device__ __forceinline__ void copy(uint32_t lds, int wave, int i0 = 0, int i1 = kDma) {
#pragma unroll
    for (int i = i0; i < i1; ++i) {
      const uint32_t to = lds + (uint32_t)(wave * kDma + i) * 1024u;
      if constexpr (ONCE)
        lds_dma16_nt(src[i], to);
      else
        lds_dma16(src[i], to);
      src[i] += advance;
    }
  }
  // A step with fewer than kBK K indices (`left`), zeros past them.  src is at that step.
  __device__ __forceinline__ void copy_last(unsigned char* lds, int wave, int lane, int left) {
    u32x4 v[kDma];
#pragma unroll
    for (int i = 0; i < kDma; ++i) {
      int row, piece;
      at(wave, lane, i, &row, &piece);
      const int keep = ALONG ? (row < left ? 8 : 0) : left - piece * 8;
      v[i] = u32x4{0, 0, 0, 0};
      if (keep > 0) v[i] = *reinterpret_cast<const u32x4*>(src[i]) & keep_mask8(keep);
    }
#pragma unroll
    for (int i = 0; i < kDma; ++i)
      *reinterpret_cast<u32x4*>(lds + (wave * kDma + i) * 1024 + lane * 16) = v[i];
  }
  // Operand of rows r .. r + 15, K 32 sub .. 32 sub + 31.  (Either form touches all 64
  // banks once per 16 or 32 lanes that the LDS serves together.)
  __device__ __forceinline__ static u32x4 read(const unsigned char* lds, int r, int sub, int lane) {
    const int i = lane & 15, g = lane >> 4;
    if constexpr (ALONG) {
      u32x4 v;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = 32 * sub + 8 * g + 4 * h + (i >> 2);
        const int at = k * (2 * R) + (((r >> 3) ^ (2 * (k & 3))) << 4) + (i & 3) * 8;
        const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s16x4*)(lds + at));
        const u32x2 w = __builtin_bit_cast(u32x2, t);
        v[2 * h] = w[0];
        v[2 * h + 1] = w[1];
      }
      return v;
    } else {
      const int row = r + i;
      return *reinterpret_cast<const u32x4*>(lds + row * 128 + (((4 * sub + g) ^ (row & 7)) << 4));
    }
  }
};

// ------------------------------------------------------------------ tiles
struct TileGrid {
  int tiles_m, tiles_n;
  int splits;            // pieces of K
  int steps;             // whole and part steps of kBK in a piece
  float* partial;        // [splits][M][n8] where splits > 1
  int64_t n8;            // N rounded up to 8
};

// A work-group's tile and its part of K.
struct Place {
  int m0, n0, split, k0, whole, left;
};
template <int BM, int BN>
__device__ __forceinline__ Place place_of(const GemmArgs& g, const TileGrid& t) {
  // tiles of one split in runs per XCD; within a run, bands of 8 rows of tiles, so that
  // the 32 tiles an XCD works on at a time share 8 rows and 4 columns of tiles in its L2
  const int tiles = t.tiles_m * t.tiles_n;
  Place p;
  p.split = (int)(blockIdx.x / (unsigned)tiles);
  const int q = xcd_runs((int)(blockIdx.x % (unsigned)tiles), tiles);
  const int band = q / (8 * t.tiles_n), in_band = q % (8 * t.tiles_n);
  const int rows = t.tiles_m - band * 8 < 8 ? t.tiles_m - band * 8 : 8;
  p.m0 = (band * 8 + in_band % rows) * BM;
  p.n0 = in_band / rows * BN;
  p.k0 = p.split * t.steps * kBK;
  const int64_t most = (int64_t)t.steps * kBK;
  const int len = g.K - p.k0 < most ? g.K - p.k0 : (int)most;
  p.whole = len / kBK;
  p.left = len % kBK;
  return p;
}

// Ends a tile: the wave's MI x NI blocks of 16 x 16 (rows m0 .., columns n0 ..) pass
// through its own part of LDS, 32 rows at a time, so that the epilogue is one loop over
// whole rows and not code for every register.  LDS rows lie four words apart in the
// banks.  All waves have done with the operands.  The residual of a pass is loaded during
// the one before: read where it was added, behind the stores of the rows before it, it
// cost 8192 x 4096 x 4096 with gelu, residual and pre 272 us instead of 257.
template <int MI, int NI>
__device__ __forceinline__ void finish(const GemmArgs& g, const TileGrid& t, int split, int m0,
                                       int n0, const f32x4 (&acc)[MI][NI], float* mine, int lane) {
  constexpr int kCols = NI * 16, kPitch = kCols + 4, kPass = 32;
  constexpr int kLanes = kCols / 8;      // of a row
  constexpr int kRows = 64 / kLanes;     // rows at once
  constexpr int kGroups = kPass / kRows;
  static_assert(MI % 2 == 0 && kPass % kRows == 0, "whole passes");
  const int n = n0 + 8 * (lane % kLanes);
  float bias[8];
  load_bias(g, n, bias);
  const bool whole = t.splits == 1;
  // the residual of a pass is on its way during the pass before it
  u32x4 q[kGroups];
#pragma unroll
  for (int i = 0; i < kGroups; ++i)
    q[i] = load_residual(g, whole ? m0 + lane / kLanes + i * kRows : g.M, n);
  for (int pass = 0; pass < MI / 2; ++pass) {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      if (i / 2 == pass) {
#pragma unroll
        for (int j = 0; j < NI; ++j)
          *reinterpret_cast<f32x4*>(mine + ((i & 1) * 16 + (lane & 15)) * kPitch + j * 16 +
                                    4 * (lane >> 4)) = acc[i][j];
      }
    }
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int r = lane / kLanes + i * kRows, m = m0 + pass * kPass + r;
      const u32x4 add = q[i];
      q[i] = load_residual(g, whole && pass + 1 < MI / 2 ? m + kPass : g.M, n);
      float v[8];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<f32x4*>(v + 4 * h) =
            *reinterpret_cast<const f32x4*>(mine + r * kPitch + 8 * (lane % kLanes) + 4 * h);
      if (m >= g.M || n >= g.N) continue;
      if (whole) {
        epilogue8(g, m, n, bias, add, v);
      } else {
        f32x4* const p =
            reinterpret_cast<f32x4*>(t.partial + ((int64_t)split * g.M + m) * t.n8 + n);
        p[0] = *reinterpret_cast<f32x4*>(v);
        p[1] = *reinterpret_cast<f32x4*>(v + 4);
      }
    }
  }
}

// Tiles of 256 x 256, eight waves of 128 x 64 each, for products with enough of them.
// Two stages of LDS.  A step has four phases (K half 0, 1) x (upper, lower half of the
// wave's rows); each reads from LDS what the next one multiplies, and the copies of the
// step after next go out in four groups over the phases: all at once, they kept the
// waves from issuing products for as long as they queued (8192 x 4096 x 4096: 214 us,
// spread 199).  Tried: 32x32x16 products (fewer instructions, but twice the
// accumulator traffic: 222 us with three places for A and two for B in LDS), five
// stages of 32 K (half lines per copy: 245), four waves of 128 x 128 (250).  256 x 128
// serves results that give 256 x 256 fewer tiles than CUs (2048 x 4096 x 4096: 63 us,
// 84 with the larger).
constexpr int kBigM = 256, kBigThreads = 512;

template <int BN, bool AK, bool BK>
__global__ __launch_bounds__(kBigThreads) void big_kernel(GemmArgs g, TileGrid t) {
  constexpr int NW = kBigThreads / 64, WN = BN / 64, WM = NW / WN;
  constexpr int MI = kBigM / WM / 16, NI = 4, MH = MI / 2;
  typedef Operand<kBigM, NW, AK> OpA;
  typedef Operand<BN, NW, BK> OpB;
  constexpr int kStage = OpA::kBytes + OpB::kBytes;
  __shared__ __attribute__((aligned(16))) unsigned char lds[2 * kStage];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const Place at = place_of<kBigM, BN>(g, t);
  const int whole = at.whole;
  OpA a;
  OpB b;
  a.init(g.A, g.lda, at.m0, g.M, at.k0, wave, lane);
  b.init(g.B, g.ldb, at.n0, g.N, at.k0, wave, lane);
  const uint32_t base = lds_addr(lds);
  f32x4 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

  // Four phases a step: (K half 0, 1) x (upper, lower half of the rows).  Each phase
  // reads from LDS what the next one multiplies; the last one reads the next step's.
  u32x4 w0[NI], w1[NI], xa[MH], xb[MH];
  auto read_w = [&](u32x4* w, const unsigned char* st, int sub) {
#pragma unroll
    for (int j = 0; j < NI; ++j) w[j] = OpB::read(st + OpA::kBytes, (wn * NI + j) * 16, sub, lane);
  };
  auto read_x = [&](u32x4* x, const unsigned char* st, int half, int sub) {
#pragma unroll
    for (int i = 0; i < MH; ++i) x[i] = OpA::read(st, (wm * MI + half * MH + i) * 16, sub, lane);
  };
  auto multiply = [&](const u32x4* w, const u32x4* x, int half) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < MH; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
        acc[half * MH + i][j] = mfma16(w[j], x[i], acc[half * MH + i][j]);
    __builtin_amdgcn_sched_barrier(0);
  };
  // A quarter of the copies of step k.
  auto group = [&](int k, int q) {
    if (k >= whole) return;
    const uint32_t to = base + (uint32_t)(k & 1) * kStage;
    constexpr int HA = OpA::kDma / 2, HB = OpB::kDma / 2;
    if (q == 0) a.copy(to, wave, 0, HA);
    if (q == 1) a.copy(to, wave, HA, 2 * HA);
    if (q == 2) b.copy(to + OpA::kBytes, wave, 0, HB);
    if (q == 3) b.copy(to + OpA::kBytes, wave, HB, 2 * HB);
  };
  auto three = [&](const unsigned char* st, int k) {
    read_x(xb, st, 1, 0);
    multiply(w0, xa, 0);
    group(k, 3);
    read_w(w1, st, 1);
    read_x(xa, st, 0, 1);
    multiply(w0, xb, 1);
    
    read_x(xb, st, 1, 1);
    multiply(w1, xa, 0);
  };
  if (whole > 0) {
    a.copy(base, wave);
    b.copy(base + OpA::kBytes, wave);
    vm_wait<0>();
    __syncthreads();
    if (whole > 1) {
      a.copy(base + kStage, wave);
      b.copy(base + kStage + OpA::kBytes, wave);
    }
    read_w(w0, lds, 0);
    read_x(xa, lds, 0, 0);
    for (int k = 0; k + 1 < whole; ++k) {
      three(lds + (k & 1) * kStage, k > 0 ? k + 1 : whole);
      lgkm_wait0();
      vm_wait<0>();                   // step k + 1 has arrived,
      __builtin_amdgcn_s_barrier();   // and step k has been read, everywhere
      asm volatile("" ::: "memory");
      const unsigned char* const next = lds + ((k + 1) & 1) * kStage;
      read_w(w0, next, 0);
      read_x(xa, next, 0, 0);
      group(k + 2, 0);
      multiply(w1, xb, 1);
      group(k + 2, 1);
      group(k + 2, 2);
    }
    three(lds + ((whole - 1) & 1) * kStage, whole);
    multiply(w1, xb, 1);
  }
  if (at.left > 0) {
    __syncthreads();
    unsigned char* const to = lds + (whole & 1) * kStage;
    a.copy_last(to, wave, lane, at.left);
    b.copy_last(to + OpA::kBytes, wave, lane, at.left);
    __syncthreads();
    read_w(w0, to, 0);
    read_x(xa, to, 0, 0);
    three(to, whole);
    multiply(w1, xb, 1);
  }

  __syncthreads();
  finish<MI, NI>(g, t, at.split, at.m0 + wm * MI * 16, at.n0 + wn * NI * 16, acc,
                 reinterpret_cast<float*>(lds + wave * (2 * kStage / NW)), lane);
  static_assert(2 * kStage / NW >= 32 * (NI * 16 + 4) * 4, "finish's rows");
}

// Smaller tiles, four waves, STAGES steps of LDS, for products with few of them: a
// step's copies are issued STAGES - 1 steps ahead and waited for by count, so that
// the memory's latency is paid once and not in every step.
// 64 x 64 with four stages and 64 x 128 with three leave room for two work-groups on a
// CU (64 x 128 with four stages has a CU to itself: 200 x 1536 to 8960 32 us, with
// three 21; 128 x 128 is no faster than 64 x 128 anywhere).  ONCE: results of one tile of
// rows, whose weights no other work-group reads, copied past the caches (64 x 1536 to
// 152064 109 -> 102 us, 32 x 4096 to 32000 57 -> 51; few_rows_kernel lost by it).
template <int BM, int BN, int WM, int WN, int STAGES, bool AK, bool BK, bool ONCE>
__global__ __launch_bounds__(WM* WN * 64) void tile_kernel(GemmArgs g, TileGrid t) {
  constexpr int NW = WM * WN, MI = BM / WM / 16, NI = BN / WN / 16;
  typedef Operand<BM, NW, AK> OpA;
  typedef Operand<BN, NW, BK> OpB;
  constexpr int kStage = OpA::kBytes + OpB::kBytes, kDma = OpA::kDma + OpB::kDma;
  __shared__ __attribute__((aligned(16))) unsigned char lds[STAGES * kStage];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const Place at = place_of<BM, BN>(g, t);
  const int whole = at.whole, steps = whole + (at.left > 0);
  OpA a;
  OpB b;
  a.init(g.A, g.lda, at.m0, g.M, at.k0, wave, lane);
  b.init(g.B, g.ldb, at.n0, g.N, at.k0, wave, lane);
  const uint32_t base = lds_addr(lds);
  f32x4 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  auto fetch = [&](int k) {
    const uint32_t to = (uint32_t)(k % STAGES) * kStage;
    if (k < whole) {
      a.copy(base + to, wave);
      b.template copy<ONCE>(base + to + OpA::kBytes, wave);
    } else if (k < steps) {
      a.copy_last(lds + to, wave, lane, at.left);
      b.copy_last(lds + to + OpA::kBytes, wave, lane, at.left);
    }
  };
#pragma unroll 1
  for (int k = 0; k < STAGES - 1; ++k) fetch(k);
#pragma unroll 1
  for (int k = 0; k < steps; ++k) {
    // step k has arrived, and step k - 1 has been read, everywhere (the counts hold while
    // every later step of the ring is one of whole copies)
    lgkm_wait0();
    if (k + STAGES - 2 < whole)
      vm_wait<(STAGES - 2) * kDma>();
    else
      vm_wait<0>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    fetch(k + STAGES - 1);
    const unsigned char* const st = lds + (k % STAGES) * kStage;
#pragma unroll
    for (int sub = 0; sub < kBK / 32; ++sub) {
      u32x4 x[MI], w[NI];
#pragma unroll
      for (int j = 0; j < NI; ++j)
        w[j] = OpB::read(st + OpA::kBytes, (wn * NI + j) * 16, sub, lane);
#pragma unroll
      for (int i = 0; i < MI; ++i) x[i] = OpA::read(st, (wm * MI + i) * 16, sub, lane);
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = mfma16(w[j], x[i], acc[i][j]);
    }
  }
  __syncthreads();
  finish<MI, NI>(g, t, at.split, at.m0 + wm * MI * 16, at.n0 + wn * NI * 16, acc,
                 reinterpret_cast<float*>(lds + wave * (STAGES * kStage / NW)), lane);
  static_assert(STAGES * kStage / NW >= 32 * (NI * 16 + 4) * 4, "finish's rows");
}

// Joins the pieces of K, in their order, and does the epilogue.
__global__ __launch_bounds__(256) void join_kernel(GemmArgs g, TileGrid t) {
  const int64_t groups = t.n8 / 8, all = groups * g.M;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all;
       i += (int64_t)gridDim.x * 256) {
    const int m = (int)(i / groups), n = (int)(i % groups) * 8;
    const float* p = t.partial + (int64_t)m * t.n8 + n;
    const u32x4 add = load_residual(g, m, n);
    f32x4 lo = *reinterpret_cast<const f32x4*>(p), hi = *reinterpret_cast<const f32x4*>(p + 4);
    for (int s = 1; s < t.splits; ++s) {
      p += (int64_t)g.M * t.n8;
      lo += *reinterpret_cast<const f32x4*>(p);
      hi += *reinterpret_cast<const f32x4*>(p + 4);
    }
    float bias[8], v[8];
    load_bias(g, n, bias);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = lo[e];
      v[4 + e] = hi[e];
    }
    epilogue8(g, m, n, bias, add, v);
  }
}

// ------------------------------------------------------------------ few rows
// Forward product of at most 16 rows: a work-group takes 16 columns (rows of W), its
// eight waves pieces of K; each lane reads W straight into the operand (16 bytes of one
// row; the second load of a pair takes the other half of its 128-byte line), eight loads
// in flight, and X likewise from the caches.  The waves' sums meet in LDS.
// 1 x 4096 to 4096: 4.0 us (weights that the caches hold), 9.7 from HBM in a row of calls.
constexpr int kFewWaves = 8;

__global__ __launch_bounds__(kFewWaves * 64) void few_rows_kernel(GemmArgs g) {
  __shared__ __attribute__((aligned(16))) float sums[kFewWaves][16][20];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, q = lane >> 4;
  const int n0 = (int)blockIdx.x * 16;
  const uint16_t* const w = g.B + (int64_t)(n0 + i < g.N ? n0 + i : g.N - 1) * g.ldb + 8 * q;
  const uint16_t* const x = g.A + (int64_t)(i < g.M ? i : g.M - 1) * g.lda + 8 * q;
  f32x4 acc{0, 0, 0, 0};
  // whole blocks of 64 K, dealt to the waves in runs
  const int blocks = g.K / 64, per = (blocks + kFewWaves - 1) / kFewWaves;
  const int b0 = wave * per < blocks ? wave * per : blocks;
  const int b1 = b0 + per < blocks ? b0 + per : blocks;
  // bias and residual of the eight results that this thread will end
  const int m = (int)threadIdx.x >> 1, n = n0 + 8 * ((int)threadIdx.x & 1);
  const bool ends = m < 16 && m < g.M && n < g.N;
  float bias[8];
  u32x4 add{0, 0, 0, 0};
  if (ends) {
    load_bias(g, n, bias);
    add = load_residual(g, m, n);
  }
  constexpr int kDeep = 4;     // blocks in flight
  for (int b = b0; b < b1; b += kDeep) {
    u32x4 wv[2 * kDeep], xv[2 * kDeep];
#pragma unroll
    for (int e = 0; e < 2 * kDeep; ++e) {
      const int k = (b + e / 2 < b1 ? b + e / 2 : b1 - 1) * 64 + (e & 1) * 32;
      wv[e] = load_bf16x8(w, k);
      xv[e] = load_bf16x8(x, k);
    }
#pragma unroll
    for (int e = 0; e < 2 * kDeep; ++e)
      if (b + e / 2 < b1) acc = mfma16(wv[e], xv[e], acc);
  }
  // the last, incomplete block, its two halves to the last two waves (one of few blocks
  // each): zeros past K on both sides
  const int k1 = blocks * 64 + (wave == kFewWaves - 1 ? 32 : 0);
  if (wave >= kFewWaves - 2 && k1 < g.K) {
    const int keep = g.K - k1 - 8 * q;
    const u32x4 mask = keep_mask8(keep);
    const int k = keep > 0 ? k1 : 0 - 8 * q;      // (a piece past the row's end: its first)
    const u32x4 wv = load_bf16x8(w, k) & mask;
    acc = mfma16(wv, load_bf16x8(x, k) & mask, acc);
  }
  // (a lane holds row i of C, columns 4 q .. 4 q + 3)
  *reinterpret_cast<f32x4*>(&sums[wave][i][4 * q]) = acc;
  __syncthreads();
  if (!ends) return;
  float v[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    f32x4 s{0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < kFewWaves; ++u)
      s += *reinterpret_cast<const f32x4*>(&sums[u][m][8 * ((int)threadIdx.x & 1) + 4 * h]);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 * h + e] = s[e];
  }
  epilogue8(g, m, n, bias, add, v);
}

// ------------------------------------------------------------------ which kernel
enum Tile { kFew, kTile64, kTile64x128, kTile256x128, kTile256 };
struct TilePlan {
  Tile tile;
  TileGrid grid;
  size_t bytes;
};
// Rows and columns of a tile, its threads, and what a step of kBK costs a work-group
// that has a CU to itself or shares it with another (us; the large tiles do not share),
// and its start and end.
struct TileKind {
  int bm, bn, threads;
  double alone, shared, ends;
};
constexpr TileKind kKinds[] = {{16, 16, 512, 0.06, 0, 0},
                               {64, 64, 256, 0.23, 0.40, 0.95},
                               {64, 128, 256, 0.44, 0.68, 1.4},
                               {256, 128, 512, 0.90, 0, 4.2},
                               {256, 256, 512, 1.45, 0, 7.3}};
constexpr int kCus = 256;

bool make_plan(Tile tile, int64_t splits, int64_t M, int64_t N, int64_t K, TilePlan* p) {
  *p = TilePlan{};
  p->tile = tile;
  const int64_t tm = (M + kKinds[tile].bm - 1) / kKinds[tile].bm;
  const int64_t tn = (N + kKinds[tile].bn - 1) / kKinds[tile].bn;
  const int64_t steps = K > 0 ? (K + kBK - 1) / kBK : 1;   // (no rows: a gradient of zeros)
  const int64_t per = (steps + splits - 1) / splits;
  splits = (steps + per - 1) / per;
  if (tm * tn * splits * kKinds[tile].threads >= (int64_t(1) << 32)) return false;
  p->grid.tiles_m = (int)tm;
  p->grid.tiles_n = (int)tn;
  p->grid.splits = (int)splits;
  p->grid.steps = (int)per;
  p->grid.n8 = round_up(N, 8);
  p->bytes = splits > 1 ? (size_t)round_up(splits * M * p->grid.n8 * 4, 256) : 0;
  return true;
}

// Estimated time (us) of `work` work-groups of `steps` steps.
double time_of(const TileKind& kind, double work, double steps) {
  if (kind.shared == 0) return ceil(work / kCus) * (steps * kind.alone + kind.ends);
  const double full = floor(work / (2 * kCus)), rest = work - full * 2 * kCus;
  const double pairs = rest > kCus ? (rest - kCus) / kCus : 0;
  return full * (steps * kind.shared + 2 * kind.ends) +
         (rest > 0 ? steps * (kind.alone + (kind.shared - kind.alone) * pairs) +
                         kind.ends * (pairs > 0 ? 2 : 1)
                   : 0);
}
// The tile and the split of K with the least estimate; a split costs the second launch
// and its pieces written and read (mostly from the caches).  Fitted on 50 products of 1
// to 8192 rows in the three forms, the kernel chosen was the fastest or within 10 % of it
// in 50 of 54 cases (the others 12 - 18 %).
bool plan_of(GemmForm form, int64_t M, int64_t N, int64_t K, TilePlan* p) {
  double least = INFINITY;
  for (int tile = kFew; tile <= kTile256; ++tile) {
    if (tile == kFew && (form != GemmForm::kForward || M > kKinds[kFew].bm)) continue;
    for (int64_t splits = 1; splits <= (tile == kFew ? 1 : 8); splits *= 2) {
      TilePlan q{};
      if (splits > 1 && K < splits * 4 * kBK) break;
      if (!make_plan((Tile)tile, splits, M, N, K, &q)) break;
      double cost = time_of(kKinds[tile],
                            (double)q.grid.tiles_m * q.grid.tiles_n * q.grid.splits, q.grid.steps);
      if (tile == kFew) cost *= 1 + (double)M / 20;
      if (q.grid.splits > 1) cost += 2.8 + (double)q.bytes * 2 / 16e6;
      if (cost < least) {
        least = cost;
        *p = q;
      }
    }
  }
  return least < INFINITY;
}


template <bool AK, bool BK>
void launch_tiles(const GemmArgs& a, const TilePlan& p, hipStream_t s) {
  const dim3 grid((unsigned)(p.grid.tiles_m * p.grid.tiles_n * p.grid.splits));
  const dim3 block((unsigned)kKinds[p.tile].threads);
  switch (p.tile) {
    case kTile64:
      if (p.grid.tiles_m == 1)
        hipLaunchKernelGGL((tile_kernel<64, 64, 2, 2, 4, AK, BK, true>), grid, block, 0, s, a,
                           p.grid);
      else
        hipLaunchKernelGGL((tile_kernel<64, 64, 2, 2, 4, AK, BK, false>), grid, block, 0, s, a,
                           p.grid);
      break;
    case kTile64x128:
      if (p.grid.tiles_m == 1)
        hipLaunchKernelGGL((tile_kernel<64, 128, 2, 2, 3, AK, BK, true>), grid, block, 0, s, a,
                           p.grid);
      else
        hipLaunchKernelGGL((tile_kernel<64, 128, 2, 2, 3, AK, BK, false>), grid, block, 0, s, a,
                           p.grid);
      break;
    case kTile256x128:
      hipLaunchKernelGGL((big_kernel<128, AK, BK>), grid, block, 0, s, a, p.grid);
      break;
    default:
      hipLaunchKernelGGL((big_kernel<256, AK, BK>), grid, block, 0, s, a, p.grid);
  }
}

// ------------------------------------------------------------------ activation gradient
// A work-group takes 8 COLS columns, its THREADS / COLS row lanes each every so manieth
// row: 256 columns and 8 lanes, or, for few rows (which one work-group then adds up alone,
// without a second launch), 16 columns and 256 lanes.
constexpr int kStripCols = 256, kRowLanes = 8, kNarrowCols = 16, kNarrowThreads = 512;

struct ActGrid {
  bool narrow;
  int rows;              // of a work-group
  int chunks;            // work-groups along T
  float* partial;        // [chunks][d], or d_bias itself
};

// Each thread takes eight columns of its rows, four rows' loads in flight.
template <int ACT, bool F32, int COLS, int THREADS>
__global__ __launch_bounds__(THREADS) void act_grad_kernel(ActGradArgs a, ActGrid t) {
  constexpr int U = 4, kLanes = THREADS / COLS, kWaves = THREADS / 64;
  __shared__ float sums[kWaves][COLS * 8];
  const int cl = (int)threadIdx.x % COLS, rl = (int)threadIdx.x / COLS;
  // (narrow strips that share lines of 128 bytes go to one L2)
  const int strip = COLS < 8 ? xcd_runs((int)blockIdx.x, (int)gridDim.x) : (int)blockIdx.x;
  const int n = (strip * COLS + cl) * 8;
  const int64_t r0 = (int64_t)blockIdx.y * t.rows;
  const int64_t r1 = r0 + t.rows < a.T ? r0 + t.rows : a.T;
  const int valid = a.d - n;
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (valid > 0) {
    for (int64_t r = r0 + rl; r < r1; r += U * kLanes) {
      u32x4 lo[U], hi[U], pre[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t row = r + u * kLanes < r1 ? r + u * kLanes : r;
        if constexpr (F32) {
          // (a row's padding ends on 16 bytes of fp32, not of eight entries)
          const u32x4* const p = reinterpret_cast<const u32x4*>(
              static_cast<const float*>(a.d_out) + row * a.ldd + n);
          lo[u] = p[0];
          hi[u] = p[valid > 4 ? 1 : 0];
        } else {
          lo[u] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.d_out) +
                                                  row * a.ldd + n);
        }
        if constexpr (ACT != kActNone)
          pre[u] = *reinterpret_cast<const u32x4*>(a.pre + row * a.ldp + n);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t row = r + u * kLanes;
        if (row >= r1) break;
        float g[8];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          if constexpr (F32) {
            g[p] = __uint_as_float(lo[u][p]);
            g[4 + p] = __uint_as_float(hi[u][p]);
          } else {
            g[2 * p] = bf16_lo(lo[u][p]);
            g[2 * p + 1] = bf16_hi(lo[u][p]);
          }
        }
        if constexpr (ACT != kActNone) {
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            g[2 * p] *= slope<ACT>(bf16_lo(pre[u][p]));
            g[2 * p + 1] *= slope<ACT>(bf16_hi(pre[u][p]));
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += g[e];
        if (a.dY != nullptr) {
          uint16_t* const p = a.dY + row * a.ldy + n;
          if (valid >= 8) {
            *reinterpret_cast<u32x4*>(p) = pack8(g);
          } else {
            for (int e = 0; e < valid; ++e) p[e] = f32_to_bf16(g[e]);
          }
        }
      }
    }
  }
  if (a.d_bias == nullptr) return;
  // the wave's row lanes, then the waves
#pragma unroll
  for (int off = COLS; off < 64; off *= 2)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] += __shfl_xor(sum[e], off);
  if ((threadIdx.x & 63) < COLS) {
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[threadIdx.x >> 6][cl * 8 + e] = sum[e];
  }
  __syncthreads();
  const int c = strip * COLS * 8 + (int)threadIdx.x;
  if (threadIdx.x >= COLS * 8 || c >= a.d) return;
  float v = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) v += sums[i][threadIdx.x];
  t.partial[(int64_t)blockIdx.y * a.d + c] = v;
}

// Adds the chunks' sums of 64 columns: four lanes a column, each every fourth chunk,
// eight loads in flight (one lane a column: 20 us for 64 chunks of 4096).
__global__ __launch_bounds__(256) void bias_join_kernel(const float* __restrict__ partial,
                                                        int chunks, int d,
                                                        float* __restrict__ out) {
  __shared__ float sums[4][64];
  const int c = (int)blockIdx.x * 64 + ((int)threadIdx.x & 63), l = (int)threadIdx.x >> 6;
  float v = 0;
  if (c < d) {
#pragma unroll 8
    for (int i = l; i < chunks; i += 4) v += partial[(int64_t)i * d + c];
  }
  sums[l][threadIdx.x & 63] = v;
  __syncthreads();
  if (l == 0 && c < d)
    out[c] = (sums[0][threadIdx.x] + sums[1][threadIdx.x]) +
             (sums[2][threadIdx.x] + sums[3][threadIdx.x]);
}

// Narrow up to 1024 rows and 640 work-groups.  With
// silu, narrow against strips and their join: 16 x 4096 3.1 us, 4.7; 501 x 1001 4.2, 6.8;
// 1024 x 4096 7.6, 8.4; 1024 x 16384 23.3, 20.5; 2048 x 4096 14.6, 13.1.  (32 columns a
// work-group: 501 x 1001 5.3, the slopes of too few CUs.)
ActGrid make_act_grid(int64_t T, int64_t d, bool sums) {
  ActGrid g{};
  g.narrow = sums && T <= 1024 && d <= 640 * kNarrowCols;
  if (g.narrow) {
    g.rows = (int)T;
    g.chunks = 1;
    return g;
  }
  const int64_t strips = (d + kStripCols - 1) / kStripCols;
  int64_t chunks = (1024 + strips - 1) / strips;
  const int64_t most = (T + kRowLanes - 1) / kRowLanes;
  if (chunks > most) chunks = most;
  if (chunks < 1) chunks = 1;
  int64_t rows = round_up((T + chunks - 1) / chunks, kRowLanes);
  if (rows < kRowLanes) rows = kRowLanes;
  g.rows = (int)(rows < (1 << 30) ? rows : 1 << 30);
  g.chunks = (int)((T + g.rows - 1) / g.rows);
  return g;
}

template <int ACT>
void launch_act(const ActGradArgs& a, const ActGrid& g, hipStream_t s) {
  const int64_t cols = g.narrow ? kNarrowCols : kStripCols;     // (d and it pass 2^31 together)
  const dim3 grid((unsigned)((a.d + cols - 1) / cols), (unsigned)g.chunks);
  const dim3 block(g.narrow ? kNarrowThreads : 256);
  constexpr int kN = kNarrowCols / 8, kS = kStripCols / 8;
  constexpr int kNT = kNarrowThreads;
  auto kernel = a.d_out_f32 ? act_grad_kernel<ACT, true, kS, 256>
                            : act_grad_kernel<ACT, false, kS, 256>;
  if (g.narrow)
    kernel = a.d_out_f32 ? act_grad_kernel<ACT, true, kN, kNT>
                         : act_grad_kernel<ACT, false, kN, kNT>;
  hipLaunchKernelGGL(kernel, grid, block, 0, s, a, g);
}

}  // namespace

size_t gemm_ws_bytes(GemmForm form, int64_t M, int64_t N, int64_t K) {
  TilePlan p{};
  return plan_of(form, M, N, K, &p) ? p.bytes : 0;
}
bool gemm_fits(GemmForm form, int64_t M, int64_t N, int64_t K) {
  TilePlan p{};
  return plan_of(form, M, N, K, &p);
}

hipError_t launch_gemm(GemmForm form, const GemmArgs& a, char* ws, hipStream_t s) {
  TilePlan p{};
  if (!plan_of(form, a.M, a.N, a.K, &p)) return hipErrorInvalidValue;
  p.grid.partial = reinterpret_cast<float*>(ws);
  if (p.tile == kFew) {
    hipLaunchKernelGGL(few_rows_kernel, dim3((unsigned)p.grid.tiles_n), dim3(kFewWaves * 64), 0, s,
                       a);
    return hipGetLastError();
  }
  switch (form) {
    case GemmForm::kForward: launch_tiles<false, false>(a, p, s); break;
    case GemmForm::kInput: launch_tiles<false, true>(a, p, s); break;
    default: launch_tiles<true, true>(a, p, s);
  }
  if (p.grid.splits > 1) {
    int64_t blocks = (p.grid.n8 / 8 * a.M + 255) / 256;
    if (blocks > 8192) blocks = 8192;
    hipLaunchKernelGGL(join_kernel, dim3((unsigned)blocks), dim3(256), 0, s, a, p.grid);
  }
  return hipGetLastError();
}

size_t act_grad_ws_bytes(int64_t T, int64_t d) {
  const ActGrid g = make_act_grid(T, d, true);
  return g.chunks > 1 ? (size_t)round_up((int64_t)g.chunks * d * 4, 256) : 0;
}

hipError_t launch_act_grad(const ActGradArgs& a, char* ws, hipStream_t s) {
  ActGrid g = make_act_grid(a.T, a.d, a.d_bias != nullptr);
  if (g.chunks < 1) g.chunks = 1;      // (no rows: the sums are zero)
  g.partial = g.chunks > 1 ? reinterpret_cast<float*>(ws) : a.d_bias;
  switch (a.act) {
    case kActNone: launch_act<kActNone>(a, g, s); break;
    case kActRelu: launch_act<kActRelu>(a, g, s); break;
    case kActSilu: launch_act<kActSilu>(a, g, s); break;
    case kActGelu: launch_act<kActGelu>(a, g, s); break;
    default: launch_act<kActGeluTanh>(a, g, s);
  }
  if (a.d_bias != nullptr && g.chunks > 1)
    hipLaunchKernelGGL(bias_join_kernel, dim3((unsigned)(((int64_t)a.d + 63) / 64)), dim3(256), 0,
                       s, g.partial, g.chunks, a.d, a.d_bias);
  return hipGetLastError();
}

}  // namespace logra
