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
//            token's values lie in the lanes of its own column and rows of other
//            policies (or holding NaN) touch nothing.  A tile's policies are
//            found by ballots; few tiles deal them to several work-groups.
//            Signs are drawn and expanded to +-1 in registers, so a seeded A is
//            never read: a decoding batch over many policies streams only U.
//   expand   out = Y + P U^T in blocks of 16 rows x 64 columns per wave, U's rows
//            as the MFMA's rows.  P (its pieces summed in order and scaled) and
//            fp32 U enter as bf16 pairs hi + lo of 16 significant bits; lo x lo,
//            2^-16 of the product, is left out.  Few blocks: one wave each
//            (adapter_block_kernel).  Many: waves walk down several with U in
//            registers (adapter_rows_kernel) or in LDS (adapter_strip_kernel).
// Bound: X and Y once in, out once (prompts); U of every policy in use, and
// launch latency (single tokens).
#include <type_traits>

#include "common.hpp"
#include "internal.hpp"
#include "policy/internal_policy.hpp"

// (a lambda that is not inlined would hold its captures in scratch memory)
#define LOGRA_INLINE __attribute__((always_inline))

namespace logra {

namespace {

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

// ---------------------------------------------------------------- project
// One work-group: kTileRows rows and a piece of k.  Its waves take 256-column
// chunks in turn and each multiplies its own with all of r, so the main loop has
// no barrier; their sums meet in LDS at the end, in order.  A chunk reaches LDS
// as two halves of 128 columns by direct global->LDS copies of whole cache lines
// (4 rows x 256 bytes an instruction), one half in flight while the other is
// multiplied; 16-byte piece j of row t lies at slot j ^ (t % 16) against bank
// conflicts.  In step s of a half, lanes 0-31 / 32-63 carry its columns 8 s ..
// / 64 + 8 s ..: byte s of one of the sign block's four words.
// 8192 x 4096 at rank 64: 18.4 us where every tile has one policy (3.6 TB/s; the
// vector unit, which expands the signs), 30 us with tiles of two among them, which
// end last.  Given bases are read again by every tile: 97 us there.  One token: 7.2
// us, latency.
constexpr int kHalfCols = 128;
constexpr int kHalfBytes = kTileRows * kHalfCols * 2;
constexpr int kRedRow = 36;   // floats of a token's 32 partial sums in LDS
constexpr int proj_waves(int nb) { return nb <= 4 ? 8 : 4; }

// Where A comes from: its seed, or memory (rows on 16-byte boundaries, or on any:
// 612 mixed rows of 33 policies, r = 100, take 44 us with k = 1040 and 83 with 1041).
enum class Basis { kSigns, kRows, kAnyRows };

// Elements col .. col + 7 of a row that lies on any boundary; `edge`: ones past k
// are not read and count as zero.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
template <bool EDGE>
__device__ __forceinline__ u32x4 load_any(const uint16_t* row, int col, int k) {
  if constexpr (!EDGE) return *reinterpret_cast<const u32x4_any*>(row + col);
  u32x4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int i = col + 2 * e;
    const uint32_t lo = row[i < k ? i : 0], hi = row[i + 1 < k ? i + 1 : 0];
    v[e] = (i < k ? lo : 0u) | (i + 1 < k ? hi << 16 : 0u);
  }
  return v;
}

// NB 32-row blocks of A.
template <int NB, Basis BASIS>
__global__ __launch_bounds__(64 * proj_waves(NB)) void adapter_project_kernel(
    AdapterArgs a, int rp, int n_split, int chunks_per_split, int n_deal, float* __restrict__ P) {
  constexpr bool GIVEN = BASIS != Basis::kSigns;
  constexpr int W = proj_waves(NB);
  // (more at once spilled registers)
  constexpr int kStepsAtOnce = BASIS == Basis::kAnyRows ? (NB >= 4 ? 1 : 2) : NB >= 4 ? 2 : 4;
  __shared__ __attribute__((aligned(16))) unsigned char stage[2][W][kHalfBytes];
  static_assert(W * kTileRows * kRedRow * 4 <= sizeof(stage), "partial sums fit");
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = tid >> 6;
  const int m = lane & 31;    // row of A in its block; token
  const int h = lane >> 5;
  const SignMasks smk = sign_masks();
  unsigned char* const buf0 = stage[0][wave];
  unsigned char* const buf1 = stage[1][wave];

  const int n_tiles = (int)((a.T + kTileRows - 1) / kTileRows);
  const int tile = (int)(blockIdx.x % n_tiles);
  const int rest = (int)(blockIdx.x / n_tiles);
  const int split = rest % n_split;
  const int deal = rest / n_split;
  const int64_t t0 = (int64_t)tile * kTileRows;
  const int all_chunks = (a.k - 1) / kChunk + 1;   // (k may end at 2^31 - 1)
  const int ch0 = split * chunks_per_split;
  const int n_chunks = min(chunks_per_split, all_chunks - ch0);
  // work-groups start at different chunks: in step they would all read the same
  // byte range of their rows, and so the same HBM channels
  const int rot = tile % n_chunks;

  Policies pol(a.adapter, t0 + lane, lane < kTileRows && t0 + lane < a.T, a.n);

  f32x16 acc[NB];
  auto clear = [&]() LOGRA_INLINE {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[b][v] = 0.0f;
  };
  auto phys = [&](int c) LOGRA_INLINE {
    c += rot;
    return ch0 + (c < n_chunks ? c : c - n_chunks);
  };
  // Rows past T re-read the last one (they belong to no policy); pieces past k
  // re-read the row's first and are cleared when read back.  (A piece that ends
  // past k is an aligned 16-byte group that holds an element of the row.)
  auto issue = [&](int c, int hc, unsigned char* dst) LOGRA_INLINE {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = 4 * i + (lane >> 4);
      const int col = c * kChunk + hc * kHalfCols + 8 * ((lane & 15) ^ (row & 15));
      const int64_t t = t0 + row < a.T ? t0 + row : a.T - 1;
      lds_dma16_nt((const void*)(a.X + t * a.ldx + (col < a.k ? col : 0)), lds_addr(dst + i * 1024));
    }
  };
  struct Signs {
    uint64_t w[NB][2];
  };
  Signs sw0, sw1;
  auto sign_words = [&](int id, int c, Signs& sw) LOGRA_INLINE {
    const uint64_t seed = a.seeds[2 * (int64_t)id], stream = a.seeds[2 * (int64_t)id + 1];
    if constexpr (NB == 1) {
      const Words4 blk = sign_block(seed, stream, (uint64_t)c, (uint64_t)m);
      sw.w[0][0] = h ? blk.w[1] : blk.w[0];
      sw.w[0][1] = h ? blk.w[3] : blk.w[2];
    } else {
      // lane half h draws the blocks of row block 2 j + h and swaps what the
      // other half needs
#pragma unroll
      for (int j = 0; j < NB / 2; ++j) {
        const Words4 blk = sign_block(seed, stream, (uint64_t)c, (uint64_t)((2 * j + h) * 32 + m));
        const uint64_t r0 = swap_halves64(h ? blk.w[0] : blk.w[1]);
        const uint64_t r2 = swap_halves64(h ? blk.w[2] : blk.w[3]);
        sw.w[2 * j][0] = h ? r0 : blk.w[0];
        sw.w[2 * j][1] = h ? r2 : blk.w[2];
        sw.w[2 * j + 1][0] = h ? blk.w[1] : r0;
        sw.w[2 * j + 1][1] = h ? blk.w[3] : r2;
      }
    }
  };
  // One half chunk: A of policy id (signs: the words at hand) against the tokens
  // with `keep` set (all bits; the others' columns get zeros).
  auto compute_cols = [&](auto edge, int id, const Signs& sw, uint32_t keep, int c, int hc,
                          const unsigned char* buf) LOGRA_INLINE {
    const int col0 = c * kChunk + hc * kHalfCols + 64 * h;
    const uint16_t* const A = GIVEN ? a.A + (int64_t)id * a.r * a.lda : nullptr;
#pragma unroll kStepsAtOnce
    for (int s = 0; s < 8; ++s) {
      const int slot = (8 * h + s) ^ (m & 15);
      u32x4 x = *reinterpret_cast<const u32x4*>(buf + m * (kHalfCols * 2) + slot * 16);
      if constexpr (decltype(edge)::value) x &= keep_mask8(a.k - (col0 + 8 * s));
      if constexpr (!GIVEN) x &= u32x4{keep, keep, keep, keep};
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        u32x4 w;
        if constexpr (GIVEN) {
          const int i = 32 * b + m;
          const uint16_t* const row = A + (int64_t)(i < a.r ? i : a.r - 1) * a.lda;
          if constexpr (BASIS == Basis::kRows)
            w = load_bf16x8_masked(row, col0 + 8 * s, a.k);
          else
            w = load_any<decltype(edge)::value>(row, col0 + 8 * s, a.k);
        } else {
          w = signs_to_bf16x8((uint32_t)(sw.w[b][hc] >> (8 * s)) & 0xFFu, smk);
        }
        acc[b] = mfma32(w, x, acc[b]);
      }
    }
  };
  auto compute = [&](int id, const Signs& sw, uint32_t keep, int c, int hc,
                     const unsigned char* buf) LOGRA_INLINE {
    if (c * kChunk > a.k - kChunk)  // the chunk that ends past k
      compute_cols(std::true_type{}, id, sw, keep, c, hc, buf);
    else
      compute_cols(std::false_type{}, id, sw, keep, c, hc, buf);
  };
  // The rows' whole piece of k, the next half chunk in flight, for all of the
  // policies dealt to this work-group (signs), or one (given bases).  The words of
  // the first two are held for both halves; those of others, rare in one tile of a
  // packed batch, are drawn for each.
  auto pass = [&](int id0, uint32_t keep0, int id1, uint32_t keep1, const Policies& more_of,
                  int u_more) LOGRA_INLINE {
    auto half = [&](int pc, int hc, const unsigned char* buf) LOGRA_INLINE {
      compute(id0, sw0, keep0, pc, hc, buf);
      if constexpr (!GIVEN) {
        if (id1 >= 0) compute(id1, sw1, keep1, pc, hc, buf);
        Policies q = more_of;
        int id;
        uint64_t rows;
        for (int u = u_more; q.next(&id, &rows); ++u) {
          if (u % n_deal != deal) continue;
          Signs sw;
          sign_words(id, pc, sw);
          compute(id, sw, ((rows >> m) & 1) ? ~0u : 0u, pc, hc, buf);
        }
      }
    };
    int c = wave;
    if (c < n_chunks) {
      issue(phys(c), 0, buf0);
      issue(phys(c), 1, buf1);
    }
    for (; c < n_chunks; c += W) {
      const int pc = phys(c);
      if constexpr (!GIVEN) {
        sign_words(id0, pc, sw0);
        if (id1 >= 0) sign_words(id1, pc, sw1);
      }
      const bool more = c + W < n_chunks;
      vm_wait<8>();          // half 0 is there; half 1's copies may be in flight
      half(pc, 0, buf0);
      if (more) {
        lgkm_wait0();        // this wave has read buf0
        issue(phys(c + W), 0, buf0);
        vm_wait<8>();        // half 1 is there
      } else {
        vm_wait<0>();
      }
      half(pc, 1, buf1);
      if (more) {
        lgkm_wait0();
        issue(phys(c + W), 1, buf1);
      }
    }
    lgkm_wait0();
  };
  // Sum of the waves, in order, and P of `rows`; the 2 W threads of a token take
  // kPer ranks each.
  auto finish = [&](uint64_t rows) LOGRA_INLINE {
    constexpr int kPer = 16 / W;
    float* const red = reinterpret_cast<float*>(&stage[0][0][0]);
    const int t = tid / (2 * W);
    const int i0 = (tid % (2 * W)) * kPer;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      __syncthreads();       // every wave is done with what lies there
#pragma unroll
      for (int v = 0; v < 16; v += 4) {
        const f32x4 q = {acc[b][v], acc[b][v + 1], acc[b][v + 2], acc[b][v + 3]};
        *reinterpret_cast<f32x4*>(red + (wave * kTileRows + m) * kRedRow + 2 * v + 4 * h) = q;
      }
      __syncthreads();
      if (((rows >> t) & 1) && 32 * b + i0 < rp) {
        float* p = P + ((int64_t)split * a.T + t0 + t) * rp + 32 * b + i0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          float sum = red[t * kRedRow + i0 + e];
#pragma unroll
          for (int w = 1; w < W; ++w) sum += red[(w * kTileRows + t) * kRedRow + i0 + e];
          // ranks past r meet no U
          p[e] = 32 * b + i0 + e < a.r ? sum : 0.0f;
        }
      }
    }
    __syncthreads();         // before the next copies
  };

  int id;
  uint64_t rows;
  if constexpr (GIVEN) {
    // (a basis may hold an infinity, whose product with a zero column is NaN:
    // one policy at a time)
    for (int u = 0; pol.next(&id, &rows); ++u) {
      if (u % n_deal != deal) continue;
      clear();
      pass(id, ~0u, -1, 0u, pol, 0);
      finish(rows);
    }
  } else {
    // Signs are finite, so the policies of a tile share its accumulators: each
    // meets the tile with the other rows zeroed.
    int ids[2] = {-1, -1};
    uint32_t keep[2] = {0, 0};
    uint64_t mine = 0;
    int n = 0, u = 0, u_more = 0;
    Policies rest = pol;
    for (; pol.next(&id, &rows); ++u) {
      if (u % n_deal != deal) continue;
      mine |= rows;
      if (n < 2) {
        ids[n] = id;
        keep[n] = ((rows >> m) & 1) ? ~0u : 0u;
        rest = pol;
        u_more = u + 1;
      }
      ++n;
    }
    if (n == 0) return;
    clear();
    // (alone in its tile: the other rows are not written)
    pass(ids[0], n == 1 ? ~0u : keep[0], ids[1], keep[1], rest, u_more);
    finish(mine);
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

// Elements K .. K + 7 of a row of U (r of them) as loaded: fp32 in both parts, bf16
// in the bits of the first.  VEC: 16-byte loads on their boundaries (r a multiple of
// 4 in fp32, of 8 in bf16); else on any, and the group that ends past r one by one.
// Past r other elements of the row stand in, which meet P's zeros there.
struct URaw {
  f32x4 v[2];
};
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
template <bool VEC>
__device__ __forceinline__ URaw load_u(const float* row, int K, int r) {
  URaw q;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = K + 4 * h;
    if constexpr (VEC) {
      q.v[h] = *reinterpret_cast<const f32x4*>(row + (at < r ? at : 0));
    } else {
      const int from = at < r ? at : 0;
      if (from + 4 <= r) {
        q.v[h] = *reinterpret_cast<const f32x4_any*>(row + from);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) q.v[h][e] = row[from + e < r ? from + e : r - 1];
      }
    }
  }
  return q;
}
template <bool VEC>
__device__ __forceinline__ URaw load_u(const uint16_t* row, int K, int r) {
  URaw q;
  if constexpr (VEC) {
    q.v[0] = *reinterpret_cast<const f32x4*>(row + (K < r ? K : 0));
  } else {
    const int from = K < r ? K : 0;
    u32x4 w;
    if (from + 8 <= r) {
      w = *reinterpret_cast<const u32x4_any*>(row + from);
    } else {
      uint32_t x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = row[from + e < r ? from + e : r - 1];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = x[2 * e] | (x[2 * e + 1] << 16);
    }
    q.v[0] = __builtin_bit_cast(f32x4, w);
  }
  return q;
}
// The pair hi, lo of loaded elements (no lo for bf16).
template <class UT>
__device__ __forceinline__ void u_pair(const URaw& q, u32x4& hi, u32x4& lo) {
  if constexpr (sizeof(UT) == 4) {
    const float x[8] = {q.v[0][0], q.v[0][1], q.v[0][2], q.v[0][3],
                        q.v[1][0], q.v[1][1], q.v[1][2], q.v[1][3]};
    split8(x, hi, lo);
  } else {
    hi = __builtin_bit_cast(u32x4, q.v[0]);
    lo = u32x4{0, 0, 0, 0};
  }
}

// The pieces of the kernels below: a wave has 16 rows x 64 columns at a time.

// P of row t at K .. K + 7 (its pieces of k added in order), scaled, as a pair.
// RP == 16 fills only the first two lane groups.
template <int RP>
__device__ __forceinline__ const float* p_at(const float* P, int64_t t, int K) {
  return P + t * RP + (RP >= 32 || K < RP ? K : 0);
}
template <int RP>
__device__ __forceinline__ void p_pair(f32x4 v0, f32x4 v1, const float* src, int64_t piece,
                                       int n_split, float sc, int K, u32x4& hi, u32x4& lo) {
  for (int i = 1; i < n_split; ++i) {
    src += piece;
    v0 += *reinterpret_cast<const f32x4*>(src);
    v1 += *reinterpret_cast<const f32x4*>(src + 4);
  }
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] = (e < 4 ? v0[e & 3] : v1[e & 3]) * sc;
    if (RP < 32) x[e] = K < RP ? x[e] : 0.0f;
  }
  split8(x, hi, lo);
}

// Orders a wave's LDS writes before its reads of what other lanes wrote.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Results cross a per-wave stage in LDS, so that Y is read and out written in
// whole 128-byte lines: 8 lanes a row, lane l columns 8 (l % 8) .. of rows l / 8
// and l / 8 + 8.
constexpr int kStageRow = 64 + 4;
__device__ __forceinline__ void stage_sums(float* stage, const f32x4* sum) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int w = 0; w < 4; ++w)
    *reinterpret_cast<f32x4*>(stage + (lane & 15) * kStageRow + 16 * w + 4 * (lane >> 4)) = sum[w];
  wave_sync();
}
// (a group that ends past d is an aligned 16 bytes that hold an element of the
// row; lanes past d re-read the row's first group and store nothing)
__device__ __forceinline__ u32x4 load_y(const AdapterArgs& a, int64_t row, int col) {
  const uint16_t* y = a.Y + (row < a.T ? row : a.T - 1) * a.ldy;
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(y + (col < a.d ? col : 0)));
}
__device__ __forceinline__ void store_out(const AdapterArgs& a, int64_t row, int col, u32x4 v) {
  uint16_t* o = a.out + row * a.ldo;
  if (col + 8 <= a.d) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(o + col));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + e < a.d) o[col + e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
  }
}
__device__ __forceinline__ u32x4 add_staged(u32x4 v, const float* stage, int r) {
  const int lane = threadIdx.x & 63;
  const f32x4 x = *reinterpret_cast<const f32x4*>(stage + r * kStageRow + 8 * (lane & 7));
  const f32x4 y = *reinterpret_cast<const f32x4*>(stage + r * kStageRow + 8 * (lane & 7) + 4);
  v[0] = pack_bf16x2(bf16_lo(v[0]) + x[0], bf16_hi(v[0]) + x[1]);
  v[1] = pack_bf16x2(bf16_lo(v[1]) + x[2], bf16_hi(v[1]) + x[3]);
  v[2] = pack_bf16x2(bf16_lo(v[2]) + y[0], bf16_hi(v[2]) + y[1]);
  v[3] = pack_bf16x2(bf16_lo(v[3]) + y[2], bf16_hi(v[3]) + y[3]);
  return v;
}

// Few rows: eight waves, one block each, of one strip of 64 columns.  The policies
// among the work-group's 128 rows, in the order of their first rows, are taken
// kSlots at a time: their U operands are brought to LDS by all waves together (the
// next ones already on their way) and each wave runs the product for those that
// occur in its block, where each row keeps its own.  A batch of many policies so
// reads a strip of each U once for 128 rows (1000 mixed tokens of eight policies,
// 4096 x 4096 at rank 64: 20 us; with each wave reading U itself 57 us).  Where
// strips alone leave CUs without work, the policies are dealt to `deal` work-groups,
// each of which writes the rows of its own (64 tokens of 33 policies at rank 100:
// 20 us, undealt 43; twice the deal 26, for every work-group reads its rows' pieces
// of P again).
constexpr int kBlockWaves = 8;

template <int RP, class UT, bool VEC>
__global__ __launch_bounds__(64 * kBlockWaves, 2) void adapter_block_kernel(
    AdapterArgs a, int n_split, float c, int deal, const float* __restrict__ P) {
  constexpr int NKS = RP < 32 ? 1 : RP / 32;
  constexpr bool kPair = sizeof(UT) == 4;
  constexpr int kParts = kPair ? 2 : 1;
  constexpr int kSlots = RP <= 32 ? 4 : RP == 64 ? 2 : 1;
  constexpr int kFrags = kSlots * NKS * 4;
  constexpr int kMine = kFrags / kBlockWaves;   // operands a wave brings
  constexpr int kOperands = kFrags * kParts * 64 * 16;
  constexpr int kStages = kBlockWaves * 16 * kStageRow * 4;
  constexpr int kRows = 16 * kBlockWaves;
  __shared__ __attribute__((aligned(16)))
  unsigned char shared[kOperands > kStages ? kOperands : kStages];
  u32x4* const us = reinterpret_cast<u32x4*>(shared);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15;
  const int g = lane >> 4;
  const int n_cb = (a.d + 63) / 64;
  const int share = (int)(blockIdx.x % deal);
  const int strip = (int)(blockIdx.x / deal);
  const int64_t rows0 = (int64_t)(strip / n_cb) * kRows;
  const int col0 = (strip % n_cb) * 64;
  const int lcol = col0 + 8 * (lane & 7);
  const int64_t row0 = rows0 + 16 * wave;
  const int64_t row = row0 + m;
  const int64_t t = row < a.T ? row : a.T - 1;

  // The policies of this work-group, one after the other: every wave walks the
  // rows' list for itself, a phase ahead, so nothing waits for the whole of it.
  auto policy_of = [&](int64_t r) LOGRA_INLINE {
    const int id = r < a.T ? a.adapter[r] : -1;
    return id < 0 || (int64_t)id >= a.n ? -1 : id;
  };
  const int id0 = policy_of(rows0 + lane), id1 = policy_of(rows0 + 64 + lane);
  u32x4 y[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) y[i] = load_y(a, row0 + (lane >> 3) + 8 * i, lcol);
  f32x4 p[NKS][2];
#pragma unroll
  for (int s = 0; s < NKS; ++s) {
    const float* src = p_at<RP>(P, t, 32 * s + 8 * g);
    p[s][0] = *reinterpret_cast<const f32x4*>(src);
    p[s][1] = *reinterpret_cast<const f32x4*>(src + 4);
  }
  uint64_t left0 = __ballot(id0 >= 0), left1 = __ballot(id1 >= 0);
  int turn = 0;
  auto next = [&]() LOGRA_INLINE {
    int id = -1;
    while (id < 0 && (left0 | left1)) {
      id = left0 ? __builtin_amdgcn_readlane(id0, __builtin_ctzll(left0))
                 : __builtin_amdgcn_readlane(id1, __builtin_ctzll(left1));
      left0 &= ~__ballot(id0 == id);
      left1 &= ~__ballot(id1 == id);
      if (turn != share) id = -1;
      turn = turn + 1 < deal ? turn + 1 : 0;
    }
    return id;
  };
  const int id_m = __shfl(wave < 4 ? id0 : id1, 16 * (wave & 3) + m);
  const float sc = id_m >= 0 ? c * a.scale[id_m] : 0.0f;
  bool own = share == 0 && id_m < 0;      // this work-group writes the row

  // Operand f of a phase: slot, step, column block.
  int cur[kSlots];
  URaw raw[kMine];
  auto bring = [&](const int* ids) LOGRA_INLINE {
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int f = wave + i * kBlockWaves;
      int id = ids[0];
#pragma unroll
      for (int j = 1; j < kSlots; ++j) id = f / (4 * NKS) == j ? ids[j] : id;
      if (id < 0) continue;
      const int col = col0 + 16 * (f & 3) + m;
      const UT* urow = static_cast<const UT*>(a.U) + (int64_t)id * a.d * a.r +
                       (int64_t)(col < a.d ? col : a.d - 1) * a.r;
      raw[i] = load_u<VEC>(urow, 32 * ((f >> 2) % NKS) + 8 * g, a.r);
    }
  };
#pragma unroll
  for (int j = 0; j < kSlots; ++j) cur[j] = next();
  bring(cur);
  // (dealt: the rest of the walk at once, so that only own rows' P are read)
  int64_t tp = t;
  if (deal > 1) {
    const uint64_t at0 = left0, at1 = left1;
    const int at_turn = turn;
#pragma unroll
    for (int j = 0; j < kSlots; ++j) own |= cur[j] >= 0 && id_m == cur[j];
    for (int id = next(); id >= 0; id = next()) own |= id_m == id;
    left0 = at0;
    left1 = at1;
    turn = at_turn;
    tp = own ? t : rows0;
  }
  u32x4 ph[NKS], pl[NKS];
  // (a piece's loads all at once: 200 rows at rank 256 in 38 us, one after the other 45)
  for (int i = 1; i < n_split; ++i) {
    f32x4 q[NKS][2];
#pragma unroll
    for (int s = 0; s < NKS; ++s) {
      const float* src = p_at<RP>(P, i * a.T + tp, 32 * s + 8 * g);
      q[s][0] = *reinterpret_cast<const f32x4*>(src);
      q[s][1] = *reinterpret_cast<const f32x4*>(src + 4);
    }
#pragma unroll
    for (int s = 0; s < NKS; ++s) {
      p[s][0] += q[s][0];
      p[s][1] += q[s][1];
    }
  }
#pragma unroll
  for (int s = 0; s < NKS; ++s)
    p_pair<RP>(p[s][0], p[s][1], nullptr, 0, 1, sc, 32 * s + 8 * g, ph[s], pl[s]);
  f32x4 sum[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) sum[w] = f32x4{0.f, 0.f, 0.f, 0.f};
  while (cur[0] >= 0) {
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int f = wave + i * kBlockWaves;
      u32x4 hi, lo;
      u_pair<UT>(raw[i], hi, lo);
      us[f * kParts * 64 + lane] = hi;
      if constexpr (kPair) us[(f * kParts + 1) * 64 + lane] = lo;
    }
    __syncthreads();
    int ahead[kSlots];
#pragma unroll
    for (int j = 0; j < kSlots; ++j) ahead[j] = next();
    bring(ahead);
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      const bool mine = cur[j] >= 0 && id_m == cur[j];
      if (__ballot(mine) == 0) continue;
      own |= mine;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < NKS; ++s) {
          const u32x4* u = us + ((j * NKS + s) * 4 + w) * kParts * 64 + lane;
          const u32x4 uh = u[0];
          v = mfma16(uh, pl[s], v);
          if constexpr (kPair) v = mfma16(u[64], ph[s], v);
          v = mfma16(uh, ph[s], v);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[w][e] = mine ? v[e] : sum[w][e];
      }
    }
    __syncthreads();     // the operands' places are free
#pragma unroll
    for (int j = 0; j < kSlots; ++j) cur[j] = ahead[j];
  }
  float* const stage = reinterpret_cast<float*>(shared) + wave * 16 * kStageRow;
  stage_sums(stage, sum);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = (lane >> 3) + 8 * i;
    const int id = __shfl(id_m, r);
    // (a row without a policy keeps its bits)
    const u32x4 v = id >= 0 ? add_staged(y[i], stage, r) : y[i];
    if (__shfl((int)own, r) && row0 + r < a.T) store_out(a, row0 + r, lcol, v);
  }
}

// Many rows, rank up to 64 and rows of U on 16-byte boundaries: four waves side by
// side along d walk down up to kRowBlocks blocks.  U's operands of the policy at
// hand stay in registers (64 at rank 64 in fp32) and are read again only where the
// policy changes; P is loaded one block ahead and Y three.  All work-groups of a
// large call are resident at once (two to a CU): with half the rows in each, the
// second half paid the first loads' latencies again.  8192 rows of 4096 at rank 64:
// 37 to 40 us in one policy, 44 to 47 in eight (the bare copy of Y in this structure
// takes 26 to 30).
constexpr int kRowBlocks = 16;

template <int RP, class UT>
__global__ __launch_bounds__(256, 2) void adapter_rows_kernel(AdapterArgs a, int n_split, float c,
                                                              int n_blocks,
                                                              const float* __restrict__ P) {
  constexpr int NKS = RP < 32 ? 1 : RP / 32;
  constexpr bool kPair = sizeof(UT) == 4;
  constexpr int kSets = kRowBlocks / 4;
  __shared__ __attribute__((aligned(16))) float stage_all[4][16 * kStageRow];
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int m = lane & 15;
  const int g = lane >> 4;
  float* const stage = stage_all[wave];
  const int n_cb = (a.d + 255) / 256;
  const int group = (int)(blockIdx.x / n_cb);
  const int col0 = (xcd_spread((int)(blockIdx.x % n_cb), group, n_cb) * 4 + wave) * 64;
  if (col0 >= a.d) return;
  const int64_t rb0 = (int64_t)group * (16 * n_blocks);
  const int lcol = col0 + 8 * (lane & 7);
  const int64_t rest = (a.T - rb0 + 15) / 16;
  const int nb = rest < n_blocks ? (int)rest : n_blocks;

  // Policies and factors of the rows, 64 to a register: a factor's address waits
  // for its policy, and so for every load issued before.
  int ids[kSets];
  float scs[kSets];
#pragma unroll
  for (int i = 0; i < kSets; ++i) {
    const int64_t row = rb0 + 64 * i + lane;
    const int id = 64 * i + lane < 16 * n_blocks && row < a.T ? a.adapter[row] : -1;
    ids[i] = id < 0 || (int64_t)id >= a.n ? -1 : id;
  }
#pragma unroll
  for (int i = 0; i < kSets; ++i) scs[i] = ids[i] >= 0 ? a.scale[ids[i]] : 0.0f;

  // Nothing may use a prefetched value before its block, or the wait comes with
  // the load.
  f32x4 p[2][NKS][2];
  u32x4 y[4][2];
  auto load_p = [&](int b, f32x4 (*q)[2]) LOGRA_INLINE {
    const int64_t row = rb0 + 16 * b + m;
#pragma unroll
    for (int s = 0; s < NKS; ++s) {
      const float* src = p_at<RP>(P, row < a.T ? row : a.T - 1, 32 * s + 8 * g);
      q[s][0] = *reinterpret_cast<const f32x4*>(src);
      q[s][1] = *reinterpret_cast<const f32x4*>(src + 4);
    }
  };
  auto load_rows = [&](int b, u32x4* v) LOGRA_INLINE {
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = load_y(a, rb0 + 16 * b + (lane >> 3) + 8 * i, lcol);
  };
  int cur = -1;
  u32x4 uh[NKS][4], ul[NKS][4];
  auto load_policy = [&](int id) LOGRA_INLINE {
    cur = id;
    const UT* U = static_cast<const UT*>(a.U) + (int64_t)id * a.d * a.r;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int col = col0 + 16 * w + m;
      const UT* urow = U + (int64_t)(col < a.d ? col : a.d - 1) * a.r;
#pragma unroll
      for (int s = 0; s < NKS; ++s)
        u_pair<UT>(load_u<true>(urow, 32 * s + 8 * g, a.r), uh[s][w], ul[s][w]);
    }
  };
  auto compute = [&](int b, const f32x4 (*q)[2], const u32x4* yv) LOGRA_INLINE {
    int id_m = ids[0];
    float sc = scs[0];
#pragma unroll
    for (int i = 1; i < kSets; ++i) {
      id_m = b >= 4 * i ? ids[i] : id_m;
      sc = b >= 4 * i ? scs[i] : sc;
    }
    id_m = __shfl(id_m, 16 * (b & 3) + m);
    sc = c * __shfl(sc, 16 * (b & 3) + m);
    const int64_t row = rb0 + 16 * b + m;
    u32x4 ph[NKS], pl[NKS];
#pragma unroll
    for (int s = 0; s < NKS; ++s) {
      const int K = 32 * s + 8 * g;
      p_pair<RP>(q[s][0], q[s][1], p_at<RP>(P, row < a.T ? row : a.T - 1, K), a.T * RP, n_split, sc,
                 K, ph[s], pl[s]);
    }
    f32x4 sum[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) sum[w] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto product = [&](int w, f32x4 v) LOGRA_INLINE {
#pragma unroll
      for (int s = 0; s < NKS; ++s) {
        v = mfma16(uh[s][w], pl[s], v);
        if constexpr (kPair) v = mfma16(ul[s][w], ph[s], v);
        v = mfma16(uh[s][w], ph[s], v);
      }
      return v;
    };
    uint64_t left = __ballot(id_m >= 0);
    if (left != 0) {
      int id = __builtin_amdgcn_readlane(id_m, __ffsll((unsigned long long)left) - 1);
      left &= ~__ballot(id_m == id);
      if (id != cur) load_policy(id);
#pragma unroll
      for (int w = 0; w < 4; ++w) sum[w] = product(w, sum[w]);
      // (rows of no policy take what they get here and drop it below)
      while (left != 0) {
        id = __builtin_amdgcn_readlane(id_m, __ffsll((unsigned long long)left) - 1);
        const bool mine = id_m == id;
        left &= ~__ballot(mine);
        load_policy(id);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const f32x4 v = product(w, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[w][e] = mine ? v[e] : sum[w][e];
        }
      }
    }
    stage_sums(stage, sum);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = (lane >> 3) + 8 * i;
      const int64_t orow = rb0 + 16 * b + r;
      const int id = __shfl(id_m, r);
      // (a row without a policy keeps its bits)
      const u32x4 added = add_staged(yv[i], stage, r);
      u32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = id >= 0 ? added[e] : yv[i][e];
      if (orow < a.T) store_out(a, orow, lcol, v);
    }
    wave_sync();
  };
  // Loads complete in the order of their issue, so a block's P goes before the Y
  // issued with it.
  load_p(0, p[0]);
#pragma unroll
  for (int j = 0; j < 3; ++j)
    if (j < nb) load_rows(j, y[j]);
  for (int b0 = 0; b0 < nb; b0 += 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int b = b0 + j;
      if (b >= nb) break;
      if (b + 1 < nb) load_p(b + 1, p[(j + 1) & 1]);
      if (b + 3 < nb) load_rows(b + 3, y[(j + 3) & 3]);
      compute(b, p[j & 1], y[j]);
    }
  }
}

// Many rows otherwise: eight waves share a strip of 64 columns and take every
// eighth of its blocks, up to kStripBlocks each.  U's operands of one policy at a
// time lie in LDS in operand order (converted once for the work-group's rows, 64
// KB at r = 256 in fp32).  A block of several policies is run for each of them, in
// turn, and each time only the rows of that one are written.  8192 rows of 4096 in
// eight policies: 84 us at rank 128, 141 at rank 256 (with each block of several
// policies reading U itself half as much again).
constexpr int kStripBlocks = 8;
constexpr int kStripWaves = 8;

template <int RP, class UT, bool VEC>
__global__ __launch_bounds__(64 * kStripWaves, 2) void adapter_strip_kernel(AdapterArgs a, int n_split, float c,
                                                            int n_blocks,
                                                            const float* __restrict__ P) {
  constexpr int NKS = RP < 32 ? 1 : RP / 32;
  constexpr bool kPair = sizeof(UT) == 4;
  constexpr int kParts = kPair ? 2 : 1;
  constexpr int kSets = kStripBlocks / 4;
  __shared__ u32x4 us[NKS * 4 * kParts * 64];
  __shared__ __attribute__((aligned(16))) float stage_all[kStripWaves][16 * kStageRow];
  __shared__ int candidate[kStripWaves];
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int m = lane & 15;
  const int g = lane >> 4;
  float* const stage = stage_all[wave];
  const int n_cb = (a.d + 63) / 64;
  const int group = (int)(blockIdx.x / n_cb);
  const int col0 = xcd_spread((int)(blockIdx.x % n_cb), group, n_cb) * 64;
  // block b of this wave starts at row rb0 + kBlockRows b
  constexpr int kBlockRows = 16 * kStripWaves;
  const int64_t rb0 = (int64_t)group * (kBlockRows * n_blocks) + 16 * wave;
  const int lcol = col0 + 8 * (lane & 7);

  // policies and factors of the wave's rows, 64 to a register
  int ids[kSets];
  float scs[kSets];
  uint64_t left[kSets], none[kSets];
#pragma unroll
  for (int i = 0; i < kSets; ++i) {
    const int b = 4 * i + (lane >> 4);
    const int64_t row = rb0 + (int64_t)kBlockRows * b + m;
    const bool in = b < n_blocks && row < a.T;
    const int id = in ? a.adapter[row] : -1;
    ids[i] = id < 0 || (int64_t)id >= a.n ? -1 : id;
    left[i] = __ballot(ids[i] >= 0);
    none[i] = __ballot(in) & ~left[i];
  }
#pragma unroll
  for (int i = 0; i < kSets; ++i) scs[i] = ids[i] >= 0 ? c * a.scale[ids[i]] : 0.0f;
  auto of_set = [&](const int b, const auto* v) {
    auto x = v[0];
#pragma unroll
    for (int i = 1; i < kSets; ++i) x = b >= 4 * i ? v[i] : x;
    return x;
  };
  // blocks (bit b) with a row in the given sets
  auto blocks_of = [&](const uint64_t* rows) {
    uint32_t need = 0;
#pragma unroll
    for (int b = 0; b < kStripBlocks; ++b)
      need |= ((rows[b / 4] >> (16 * (b & 3))) & 0xFFFFu) ? 1u << b : 0u;
    return need;
  };
  if (a.out != a.Y) {      // rows without a policy are copied
    for (uint32_t need = blocks_of(none); need; need &= need - 1) {
      const int b = __builtin_ctz(need);
      const uint32_t rows = (uint32_t)(of_set(b, none) >> (16 * (b & 3)));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = (lane >> 3) + 8 * i;
        const int64_t row = rb0 + kBlockRows * b + r;
        const u32x4 v = load_y(a, row, lcol);
        if ((rows >> r) & 1) store_out(a, row, lcol, v);
      }
    }
  }

  for (;;) {
    // the work-group's next policy: the first one left in its first wave with any
    int next = -1;
#pragma unroll
    for (int i = kSets - 1; i >= 0; --i)
      if (left[i])
        next = __builtin_amdgcn_readlane(ids[i], __ffsll((unsigned long long)left[i]) - 1);
    if (lane == 0) candidate[wave] = next;
    __syncthreads();       // (and every wave is done with us)
    int id = -1;
#pragma unroll
    for (int w = kStripWaves - 1; w >= 0; --w) id = candidate[w] >= 0 ? candidate[w] : id;
    if (id < 0) break;
    const UT* U = static_cast<const UT*>(a.U) + (int64_t)id * a.d * a.r;
    for (int f = wave; f < 4 * NKS; f += kStripWaves) {   // an operand (s, w) a wave
      const int s = f >> 2;
      const int col = col0 + 16 * (f & 3) + m;
      u32x4 hi, lo;
      u_pair<UT>(load_u<VEC>(U + (int64_t)(col < a.d ? col : a.d - 1) * a.r, 32 * s + 8 * g, a.r),
                 hi, lo);
      us[f * kParts * 64 + lane] = hi;
      if constexpr (kPair) us[(f * kParts + 1) * 64 + lane] = lo;
    }
    __syncthreads();

    uint64_t mine[kSets];
#pragma unroll
    for (int i = 0; i < kSets; ++i) {
      mine[i] = __ballot(ids[i] == id);
      left[i] &= ~mine[i];
    }
    uint32_t need = blocks_of(mine);
    const int nb = __builtin_popcount(need);
    uint32_t order = 0;    // four bits for each block to do
    for (int j = 0; need; ++j, need &= need - 1) order |= (uint32_t)__builtin_ctz(need) << (4 * j);

    f32x4 p[2][NKS][2];
    u32x4 y[4][2];
    auto load_p = [&](int b, f32x4 (*q)[2]) LOGRA_INLINE {
      const int64_t row = rb0 + kBlockRows * b + m;
#pragma unroll
      for (int s = 0; s < NKS; ++s) {
        const float* src = p_at<RP>(P, row < a.T ? row : a.T - 1, 32 * s + 8 * g);
        q[s][0] = *reinterpret_cast<const f32x4*>(src);
        q[s][1] = *reinterpret_cast<const f32x4*>(src + 4);
      }
    };
    auto load_rows = [&](int b, u32x4* v) LOGRA_INLINE {
#pragma unroll
      for (int i = 0; i < 2; ++i) v[i] = load_y(a, rb0 + kBlockRows * b + (lane >> 3) + 8 * i, lcol);
    };
    auto compute = [&](int b, const f32x4 (*q)[2], const u32x4* yv) LOGRA_INLINE {
      const float sc = __shfl(of_set(b, scs), 16 * (b & 3) + m);
      const int64_t row = rb0 + kBlockRows * b + m;
      f32x4 sum[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) sum[w] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < NKS; ++s) {
        const int K = 32 * s + 8 * g;
        const float* src = p_at<RP>(P, row < a.T ? row : a.T - 1, K);
        u32x4 ph, pl;
        p_pair<RP>(q[s][0], q[s][1], src, a.T * RP, n_split, sc, K, ph, pl);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const u32x4 uh = us[((s * 4 + w) * kParts) * 64 + lane];
          sum[w] = mfma16(uh, pl, sum[w]);
          if constexpr (kPair)
            sum[w] = mfma16(us[((s * 4 + w) * kParts + 1) * 64 + lane], ph, sum[w]);
          sum[w] = mfma16(uh, ph, sum[w]);
        }
      }
      stage_sums(stage, sum);
      const uint32_t rows = (uint32_t)(of_set(b, mine) >> (16 * (b & 3)));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = (lane >> 3) + 8 * i;
        const u32x4 v = add_staged(yv[i], stage, r);
        if ((rows >> r) & 1) store_out(a, rb0 + kBlockRows * b + r, lcol, v);
      }
      wave_sync();
    };
    // Loads complete in the order of their issue, so a block's P goes before the
    // Y issued with it.
    auto block = [&](int j) { return (int)((order >> (4 * j)) & 15u); };
    if (nb > 0) load_p(block(0), p[0]);
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (j < nb) load_rows(block(j), y[j]);
    for (int j0 = 0; j0 < nb; j0 += 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = j0 + i;
        if (j >= nb) break;
        if (j + 1 < nb) load_p(block(j + 1), p[(i + 1) & 1]);
        if (j + 3 < nb) load_rows(block(j + 3), y[(i + 3) & 3]);
        compute(block(j), p[i & 1], y[i]);
      }
    }
  }
}

// ---------------------------------------------------------------- launches
constexpr int64_t kCus = 256;

template <int RP>
void launch_project(const AdapterArgs& a, const AdapterPlan& p, float* P, hipStream_t s) {
  constexpr int NB = RP < 32 ? 1 : RP / 32;
  const int64_t tiles = (a.T + kTileRows - 1) / kTileRows;
  const int64_t base = tiles * p.n_split;
  int64_t deal = kCus / base;
  if (deal < 1) deal = 1;
  if (deal > kTileRows) deal = kTileRows;
  if (deal > a.n) deal = a.n;
  const dim3 grid((unsigned)(base * deal)), block(64 * proj_waves(NB));
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, s, a, RP, p.n_split, p.chunks_per_split, (int)deal,
                       P);
  };
  if (!a.A)
    launch(adapter_project_kernel<NB, Basis::kSigns>);
  else if (a.lda % 8 == 0 && (reinterpret_cast<uintptr_t>(a.A) & 15) == 0)
    launch(adapter_project_kernel<NB, Basis::kRows>);
  else
    launch(adapter_project_kernel<NB, Basis::kAnyRows>);
}

template <int RP, class UT, bool VEC>
void launch_expand(const AdapterArgs& a, const AdapterPlan& p, float c, const float* P,
                   hipStream_t s) {
  const int64_t n_cb = (a.d + 63) / 64;
  const int64_t blocks = (a.T + 15) / 16;
  // Eight blocks to a SIMD and more: walk down several with one U.  Both launches of
  // a call, 4096 x 4096, eight policies, us here / by the block kernel:
  //   rank 64     2047 rows in runs  42 /  37, mixed 141 /  60; 4096: 60 /  57, 270 / 108
  //   rank 256    2047 rows in runs 156 / 121, mixed 531 / 190; 4096: 159 / 160, 616 / 315
  //   rank 16     2047 rows in runs  23 /  24, mixed  36 /  34; 4096: 38 /  38,  66 /  60
  // so in runs the two meet near 4096 rows, and batches that mix policies would be
  // faster by blocks past that too.
  if (blocks * n_cb >= 8 * 4 * kCus) {
    if constexpr (RP <= 64 && VEC) {
      const int64_t wide = (a.d + 255) / 256;
      int64_t per = (blocks * wide + 2 * kCus - 1) / (2 * kCus);   // two work-groups to a CU
      per = per < 1 ? 1 : per > kRowBlocks ? kRowBlocks : per;
      hipLaunchKernelGGL((adapter_rows_kernel<RP, UT>),
                         dim3((unsigned)((blocks + per - 1) / per * wide)), dim3(256), 0, s, a,
                         p.n_split, c, (int)per, P);
    } else {
      int64_t per = blocks * n_cb / (kStripWaves * kCus);
      per = per < 1 ? 1 : per > kStripBlocks ? kStripBlocks : per;
      const int64_t rows = kStripWaves * per;
      hipLaunchKernelGGL((adapter_strip_kernel<RP, UT, VEC>),
                         dim3((unsigned)((blocks + rows - 1) / rows * n_cb)),
                         dim3(64 * kStripWaves), 0, s, a, p.n_split, c, (int)per, P);
    }
    return;
  }
  const int64_t base = (blocks + kBlockWaves - 1) / kBlockWaves * n_cb;
  int64_t deal = 2 * kCus / base;
  if (deal > a.n) deal = a.n;
  if (deal > a.T) deal = a.T;
  if (deal < 1) deal = 1;
  hipLaunchKernelGGL((adapter_block_kernel<RP, UT, VEC>), dim3((unsigned)(base * deal)),
                     dim3(64 * kBlockWaves), 0, s, a, p.n_split, c, (int)deal, P);
}

template <int RP>
void launch_both(const AdapterArgs& a, bool u_f32, const AdapterPlan& p, float c, float* P,
                 hipStream_t s) {
  launch_project<RP>(a, p, P, s);
  const bool vec = a.r % (u_f32 ? 4 : 8) == 0 && (reinterpret_cast<uintptr_t>(a.U) & 15) == 0;
  if (u_f32) {
    if (vec)
      launch_expand<RP, float, true>(a, p, c, P, s);
    else
      launch_expand<RP, float, false>(a, p, c, P, s);
  } else {
    if (vec)
      launch_expand<RP, uint16_t, true>(a, p, c, P, s);
    else
      launch_expand<RP, uint16_t, false>(a, p, c, P, s);
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
  // pieces of k while tiles leave CUs without one (a work-group has a CU's LDS
  // to itself), each with a chunk for every wave
  const int64_t waves = proj_waves(p->rp / 32);
  int64_t split = (kCus + tiles - 1) / tiles;
  if (split > (chunks + waves - 1) / waves) split = (chunks + waves - 1) / waves;
  if (split > 8) split = 8;
  const int64_t per = (chunks + split - 1) / split;
  p->chunks_per_split = (int)per;
  p->n_split = (int)((chunks + per - 1) / per);
  p->total = (size_t)round_up((int64_t)p->n_split * T * p->rp * 4, 256);
  // (flat grids: work-groups, and threads below 2^32)
  const int64_t most = (int64_t(1) << 24) - 1;
  return tiles * p->n_split <= most / 2 &&                                     // project
         (T + 255) / 256 * ((d + 255) / 256) <= most &&                        // rows
         (T + 1023) / 1024 * ((d + 63) / 64) <= most / 2;                      // strip
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
