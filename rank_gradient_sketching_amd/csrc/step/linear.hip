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
#include <math.h>

#include "common.hpp"
#include "internal.hpp"
#include "step/internal_step.hpp"

namespace logra {

namespace {

constexpr int kBK = 64;         // K of one step

typedef short s16x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ activations
template <int ACT>
__device__ __forceinline__ float activate(float x) {
  if constexpr (ACT == kActRelu) return x > 0.f || x != x ? x : 0.f;
  if constexpr (ACT == kActSilu) return x / (1.f + __expf(-x));
  // (erfc keeps the digits of Phi where 1 + erf would cancel)
  if constexpr (ACT == kActGelu) return 0.5f * x * erfcf(x * -0.70710678118654752f);
  if constexpr (ACT == kActGeluTanh) {
    const float y = 1.5957691216057308f * fmaf(0.044715f * x * x, x, x);
    return x / (1.f + __expf(-y));
  }
  return x;
}
template <int ACT>
__device__ __forceinline__ float slope(float x) {
  // (from 100 on the slope is 0 or 1 in fp32, and no product below is inf times 0)
  if (fabsf(x) > 100.f) x = copysignf(100.f, x);
  if constexpr (ACT == kActRelu) return x > 0.f ? 1.f : x != x ? x : 0.f;
  if constexpr (ACT == kActSilu) {
    const float s = 1.f / (1.f + __expf(-x)), r = 1.f / (1.f + __expf(x));
    return s * fmaf(x, r, 1.f);
  }
  if constexpr (ACT == kActGelu)
    return fmaf(x * 0.39894228040143268f, __expf(-0.5f * x * x),
                0.5f * erfcf(x * -0.70710678118654752f));
  if constexpr (ACT == kActGeluTanh) {
    const float x2 = x * x;
    const float y = 1.5957691216057308f * fmaf(0.044715f * x2, x, x);
    const float dy = 1.5957691216057308f * fmaf(3.f * 0.044715f, x2, 1.f);
    const float s = 1.f / (1.f + __expf(-y)), r = 1.f / (1.f + __expf(y));
    return s * fmaf(x * dy, r, 1.f);
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
// Four consecutive columns n .. n + 3 of row m, n a multiple of 4.
__device__ __forceinline__ void epilogue4(const GemmArgs& g, int m, int n, f32x4 v) {
  const int valid = g.N - n;
  if (valid <= 0) return;
  if (g.bias != nullptr) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < valid)
        v[e] += g.bias_f32 ? static_cast<const float*>(g.bias)[n + e]
                           : bf16_to_f32(static_cast<const uint16_t*>(g.bias)[n + e]);
  }
  if (g.pre != nullptr) {
    uint16_t* const p = g.pre + (int64_t)m * g.ldpre + n;
    if (valid >= 4) {
      *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    } else {
      for (int e = 0; e < valid; ++e) p[e] = f32_to_bf16(v[e]);
    }
  }
  if (g.act != kActNone) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = activate_any(v[e], g.act);
  }
  if (g.add != nullptr) {
    const uint16_t* const p = g.add + (int64_t)m * g.ldadd + n;
    if (valid >= 4) {
      const u32x2 q = *reinterpret_cast<const u32x2*>(p);
      v += f32x4{bf16_lo(q[0]), bf16_hi(q[0]), bf16_lo(q[1]), bf16_hi(q[1])};
    } else {
      for (int e = 0; e < valid; ++e) v[e] += bf16_to_f32(p[e]);
    }
  }
  if (g.c_f32) {
    float* const p = static_cast<float*>(g.C) + (int64_t)m * g.ldc + n;
    if (valid >= 4) {
      f32x4* const q = reinterpret_cast<f32x4*>(p);
      *q = g.accumulate ? *q + v : v;
    } else {
      for (int e = 0; e < valid; ++e) p[e] = g.accumulate ? p[e] + v[e] : v[e];
    }
  } else {
    uint16_t* const p = static_cast<uint16_t*>(g.C) + (int64_t)m * g.ldc + n;
    if (valid >= 4) {
      *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
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
  __device__ __forceinline__ void copy(uint32_t lds, int wave) {
#pragma unroll
    for (int i = 0; i < kDma; ++i) {
      lds_dma16(src[i], lds + (uint32_t)(wave * kDma + i) * 1024u);
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
  // Operand of rows r .. r + 15, K 32 sub .. 32 sub + 31.
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
  float* partial;        // [splits][M][N4] where splits > 1
  int64_t n4;            // N rounded up to 4
};

template <int BM, int BN, int WM, int WN, bool AK, bool BK>
__global__ __launch_bounds__(WM* WN * 64) void tile_kernel(GemmArgs g, TileGrid t) {
  constexpr int NW = WM * WN;
  constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
  typedef Operand<BM, NW, AK> OpA;
  typedef Operand<BN, NW, BK> OpB;
  constexpr int kStage = OpA::kBytes + OpB::kBytes;
  __shared__ __attribute__((aligned(16))) unsigned char lds[2 * kStage];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  // tiles of one split in runs per XCD; within a run, bands of 8 rows of tiles
  const int tiles = t.tiles_m * t.tiles_n;
  const int split = (int)blockIdx.x / tiles;
  const int q = xcd_runs((int)blockIdx.x % tiles, tiles);
  const int band = q / (8 * t.tiles_n), in_band = q % (8 * t.tiles_n);
  const int rows = t.tiles_m - band * 8 < 8 ? t.tiles_m - band * 8 : 8;
  const int tm = band * 8 + in_band % rows, tn = in_band / rows;
  const int m0 = tm * BM, n0 = tn * BN;
  const int k0 = split * t.steps * kBK;
  const int k_end = k0 + t.steps * kBK < g.K ? k0 + t.steps * kBK : g.K;
  const int whole = (k_end - k0) / kBK, left = (k_end - k0) % kBK;

  OpA a;
  OpB b;
  a.init(g.A, g.lda, m0, g.M, k0, wave, lane);
  b.init(g.B, g.ldb, n0, g.N, k0, wave, lane);
  const uint32_t base = lds_addr(lds);
  f32x4 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

  auto step = [&](const unsigned char* st) {
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
  };
  if (whole > 0) {
    a.copy(base, wave);
    b.copy(base + OpA::kBytes, wave);
  }
  for (int k = 0; k < whole; ++k) {
    vm_wait<0>();
    __syncthreads();      // step k has arrived, and step k - 1 has been read, everywhere
    if (k + 1 < whole) {
      const uint32_t to = base + (uint32_t)((k + 1) & 1) * kStage;
      a.copy(to, wave);
      b.copy(to + OpA::kBytes, wave);
    }
    step(lds + (k & 1) * kStage);
  }
  if (left > 0) {
    __syncthreads();
    unsigned char* const to = lds + (whole & 1) * kStage;
    a.copy_last(to, wave, lane, left);
    b.copy_last(to + OpA::kBytes, wave, lane, left);
    __syncthreads();
    step(to);
  }

  // The wave's results pass through LDS, 32 rows at a time, so that the epilogue is one
  // loop over whole rows (16 lanes a row, four rows at once) and not code for every
  // register.  Rows lie four words apart in the banks.
  constexpr int kCols = NI * 16, kPitch = kCols + 4, kPass = 32;
  static_assert(kPass * kPitch * 4 <= 2 * kStage / NW && kCols == 64 && MI % 2 == 0, "fits");
  __syncthreads();
  float* const mine = reinterpret_cast<float*>(lds + wave * (2 * kStage / NW));
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
    const int n = n0 + wn * kCols + 4 * (lane & 15);
    for (int r = lane >> 4; r < kPass; r += 4) {
      const int m = m0 + (wm * MI + 2 * pass) * 16 + r;
      const f32x4 v = *reinterpret_cast<const f32x4*>(mine + r * kPitch + 4 * (lane & 15));
      if (m >= g.M || n >= g.N) continue;
      if (t.splits == 1)
        epilogue4(g, m, n, v);
      else
        *reinterpret_cast<f32x4*>(t.partial + ((int64_t)split * g.M + m) * t.n4 + n) = v;
    }
  }
}

// Joins the pieces of K, in their order, and does the epilogue.
__global__ __launch_bounds__(256) void join_kernel(GemmArgs g, TileGrid t) {
  const int64_t quads = t.n4 / 4, all = quads * g.M;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all;
       i += (int64_t)gridDim.x * 256) {
    const int m = (int)(i / quads), n = (int)(i % quads) * 4;
    const float* p = t.partial + (int64_t)m * t.n4 + n;
    f32x4 v = *reinterpret_cast<const f32x4*>(p);
    for (int s = 1; s < t.splits; ++s) {
      p += (int64_t)g.M * t.n4;
      v += *reinterpret_cast<const f32x4*>(p);
    }
    epilogue4(g, m, n, v);
  }
}

struct TilePlan {
  int bm, bn;
  TileGrid grid;
  size_t bytes;
};

TilePlan make_tile_plan(int64_t M, int64_t N, int64_t K) {
  TilePlan p{};
  p.bm = 128;
  p.bn = 128;
  const int64_t tm = (M + p.bm - 1) / p.bm, tn = (N + p.bn - 1) / p.bn;
  const int64_t steps = K > 0 ? (K + kBK - 1) / kBK : 1;   // (no rows: a gradient of zeros)
  int64_t splits = tm * tn >= 256 ? 1 : 512 / (tm * tn);
  if (splits > steps / 4) splits = steps / 4;
  if (splits < 1) splits = 1;
  const int64_t per = (steps + splits - 1) / splits;
  splits = (steps + per - 1) / per;
  p.grid.tiles_m = (int)tm;
  p.grid.tiles_n = (int)tn;
  p.grid.splits = (int)splits;
  p.grid.steps = (int)per;
  p.grid.n4 = (N + 3) / 4 * 4;
  p.bytes = splits > 1 ? (size_t)round_up(splits * M * p.grid.n4 * 4, 256) : 0;
  return p;
}

template <bool AK, bool BK>
void launch_tiles(const GemmArgs& a, const TilePlan& p, hipStream_t s) {
  const dim3 grid((unsigned)(p.grid.tiles_m * p.grid.tiles_n * p.grid.splits));
  hipLaunchKernelGGL((tile_kernel<128, 128, 2, 2, AK, BK>), grid, dim3(256), 0, s, a, p.grid);
}

// ------------------------------------------------------------------ activation gradient
constexpr int kColThreads = 32, kRowLanes = 8;     // a work-group: 256 columns
constexpr int kStripCols = kColThreads * 8;

struct ActGrid {
  int rows;              // of a work-group
  int chunks;            // work-groups along T
  float* partial;        // [chunks][d], or d_bias itself
};

template <int ACT, bool F32>
__global__ __launch_bounds__(256) void act_grad_kernel(ActGradArgs a, ActGrid t) {
  __shared__ float sums[kRowLanes][kStripCols];
  const int cl = (int)threadIdx.x % kColThreads, rl = (int)threadIdx.x / kColThreads;
  const int n = ((int)blockIdx.x * kColThreads + cl) * 8;
  const int64_t r0 = (int64_t)blockIdx.y * t.rows;
  const int64_t r1 = r0 + t.rows < a.T ? r0 + t.rows : a.T;
  const int valid = a.d - n;
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (valid > 0) {
    for (int64_t r = r0 + rl; r < r1; r += kRowLanes) {
      float g[8];
      if constexpr (F32) {
        // (the row's padding ends on 16 bytes of fp32, not of eight entries)
        const float* const p = static_cast<const float*>(a.d_out) + r * a.ldd + n;
        const f32x4 lo = *reinterpret_cast<const f32x4*>(p);
        f32x4 hi{0, 0, 0, 0};
        if (valid > 4) hi = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          g[e] = lo[e];
          g[4 + e] = hi[e];
        }
      } else {
        const u32x4 q = *reinterpret_cast<const u32x4*>(
            static_cast<const uint16_t*>(a.d_out) + r * a.ldd + n);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          g[2 * p] = bf16_lo(q[p]);
          g[2 * p + 1] = bf16_hi(q[p]);
        }
      }
      if constexpr (ACT != kActNone) {
        const u32x4 q = *reinterpret_cast<const u32x4*>(a.pre + r * a.ldp + n);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          g[2 * p] *= slope<ACT>(bf16_lo(q[p]));
          g[2 * p + 1] *= slope<ACT>(bf16_hi(q[p]));
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += g[e];
      if (a.dY != nullptr) {
        uint16_t* const p = a.dY + r * a.ldy + n;
        if (valid >= 8) {
          u32x4 y;
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = pack_bf16x2(g[2 * e], g[2 * e + 1]);
          *reinterpret_cast<u32x4*>(p) = y;
        } else {
          for (int e = 0; e < valid; ++e) p[e] = f32_to_bf16(g[e]);
        }
      }
    }
  }
  if (a.d_bias == nullptr) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[rl][cl * 8 + e] = sum[e];
  __syncthreads();
  const int c = (int)blockIdx.x * kStripCols + (int)threadIdx.x;
  if (c >= a.d) return;
  float v = 0;
#pragma unroll
  for (int i = 0; i < kRowLanes; ++i) v += sums[i][threadIdx.x];
  t.partial[(int64_t)blockIdx.y * a.d + c] = v;
}

__global__ __launch_bounds__(256) void bias_join_kernel(const float* __restrict__ partial,
                                                        int chunks, int d,
                                                        float* __restrict__ out) {
  const int c = (int)blockIdx.x * 256 + (int)threadIdx.x;
  if (c >= d) return;
  float v = 0;
  for (int i = 0; i < chunks; ++i) v += partial[(int64_t)i * d + c];
  out[c] = v;
}

ActGrid make_act_grid(int64_t T, int64_t d) {
  ActGrid g{};
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
  const dim3 grid((unsigned)((a.d + kStripCols - 1) / kStripCols), (unsigned)g.chunks);
  if (a.d_out_f32)
    hipLaunchKernelGGL((act_grad_kernel<ACT, true>), grid, dim3(256), 0, s, a, g);
  else
    hipLaunchKernelGGL((act_grad_kernel<ACT, false>), grid, dim3(256), 0, s, a, g);
}

}  // namespace

size_t gemm_ws_bytes(GemmForm, int64_t M, int64_t N, int64_t K) {
  return make_tile_plan(M, N, K).bytes;
}

hipError_t launch_gemm(GemmForm form, const GemmArgs& a, char* ws, hipStream_t s) {
  TilePlan p = make_tile_plan(a.M, a.N, a.K);
  p.grid.partial = reinterpret_cast<float*>(ws);
  switch (form) {
    case GemmForm::kForward: launch_tiles<false, false>(a, p, s); break;
    case GemmForm::kInput: launch_tiles<false, true>(a, p, s); break;
    default: launch_tiles<true, true>(a, p, s);
  }
  if (p.grid.splits > 1) {
    int64_t blocks = (p.grid.n4 / 4 * a.M + 255) / 256;
    if (blocks > 8192) blocks = 8192;
    hipLaunchKernelGGL(join_kernel, dim3((unsigned)blocks), dim3(256), 0, s, a, p.grid);
  }
  return hipGetLastError();
}

size_t act_grad_ws_bytes(int64_t T, int64_t d) {
  const ActGrid g = make_act_grid(T, d);
  return g.chunks > 1 ? (size_t)round_up((int64_t)g.chunks * d * 4, 256) : 0;
}

hipError_t launch_act_grad(const ActGradArgs& a, char* ws, hipStream_t s) {
  ActGrid g = make_act_grid(a.T, a.d);
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
    hipLaunchKernelGGL(bias_join_kernel, dim3((unsigned)((a.d + 255) / 256)), dim3(256), 0, s,
                       g.partial, g.chunks, a.d, a.d_bias);
  return hipGetLastError();
}

}  // namespace logra
