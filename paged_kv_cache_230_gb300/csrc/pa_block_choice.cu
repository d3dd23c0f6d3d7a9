// Choosing the blocks a decode step attends to: the bounds of each block's
// keys, their scores against the step's queries, and the selection.
#include <math_constants.h>

#include <type_traits>

#include "pa_launch.h"
#include "pa_pdl.cuh"
#include "pa_ptx.cuh"
#include "pa_row_quant.cuh"
#include "pagedattn.h"

namespace pa {

namespace {

enum : int { kF16c = PA_F16, kBF16c = PA_BF16, kE4M3c = PA_FP8_E4M3 };

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Eight cache values at element index `at` (a multiple of 8) as they lie, and
// as four pairs of 16 bits (E4M3 widened to f16, exactly).
template <int KV>
using Raw8 = std::conditional_t<KV == kE4M3c, uint2, uint4>;

template <int KV>
__device__ __forceinline__ Raw8<KV> load8(const void* base, int64_t at) {
  return load_written(reinterpret_cast<const Raw8<KV>*>(static_cast<const uint8_t*>(base) + at * (KV == kE4M3c ? 1 : 2)));
}

template <int KV>
__device__ __forceinline__ void pairs8(const Raw8<KV>& u, uint32_t (&w)[4]) {
  if constexpr (KV == kE4M3c) {
    e4m3x4_to_f16x2x2(u.x, w[0], w[1]);
    e4m3x4_to_f16x2x2(u.y, w[2], w[3]);
  } else {
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  }
}

// The inverse, for values that were loaded so (E4M3 rounds nothing).
template <int KV>
__device__ __forceinline__ void store8(void* base, int64_t at, const uint32_t (&w)[4]) {
  if constexpr (KV == kE4M3c) {
    uint32_t c[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2_raw h = *reinterpret_cast<const __half2_raw*>(&w[i]);
      c[i / 2] |= static_cast<uint32_t>(__nv_cvt_halfraw2_to_fp8x2(h, __NV_SATFINITE, __NV_E4M3)) << (16 * (i & 1));
    }
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + at) = make_uint2(c[0], c[1]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The larger (HIGH) or smaller of each half of two pairs, NaN if either is.
template <bool BF16, bool HIGH>
__device__ __forceinline__ uint32_t pair_extreme(uint32_t a, uint32_t b) {
  if constexpr (BF16) {
    const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&a);
    const __nv_bfloat162 y = *reinterpret_cast<const __nv_bfloat162*>(&b);
    const __nv_bfloat162 z = HIGH ? __hmax2_nan(x, y) : __hmin2_nan(x, y);
    return *reinterpret_cast<const uint32_t*>(&z);
  } else {
    const __half2 x = *reinterpret_cast<const __half2*>(&a);
    const __half2 y = *reinterpret_cast<const __half2*>(&b);
    const __half2 z = HIGH ? __hmax2_nan(x, y) : __hmin2_nan(x, y);
    return *reinterpret_cast<const uint32_t*>(&z);
  }
}

__device__ __forceinline__ int clamped_length(const int32_t* lens, int64_t i, int lmax, int* err) {
  const int L = lens[i];
  if (L < 0 || L > lmax) {
    if (threadIdx.x == 0) atomicOr(err, PA_DEVERR_CONTEXT_LEN);
    return min(max(L, 0), lmax);
  }
  return L;
}

// ---- bounds -----------------------------------------------------------------
// CTA = (sequence, one of its newest blocks): a thread per eight channels of a
// kv head reads the block's live keys and keeps their least and largest, two to
// a register in the keys' own type.  After a decode step it is one small launch:
// the newest blocks of 8 sequences of 8 heads of 128 take 2.7 us, of which the
// launch is 2 (the keys one at a time, in float32: 3.5).
template <int KV>
__global__ void __launch_bounds__(128) block_bounds_kernel(const BoundsParams p) {
  pdl_enter();
  const int s = blockIdx.x / p.touched;
  const int L = clamped_length(p.context_lens, s, p.maxB * p.bs, p.err);
  const int j = max(L - p.num_new, 0) / p.bs + blockIdx.x % p.touched;
  const int live = min(p.bs, L - j * p.bs);
  if (live <= 0) return;
  const int b = load_written(p.block_tables + static_cast<int64_t>(s) * p.maxB + j);
  if (b < 0 || b >= p.num_blocks) {
    if (threadIdx.x == 0) atomicOr(p.err, PA_DEVERR_BLOCK_ID);
    return;
  }
  const int pieces = p.D / 8;
  for (int i = threadIdx.x; i < p.Hkv * pieces; i += blockDim.x) {
    const int h = i / pieces, c = i % pieces;
    const int64_t row0 = (static_cast<int64_t>(b) * p.Hkv + h) * p.bs;
    uint32_t lo[4], hi[4];
    // eight loads at a time whatever the block holds: rows past the last live
    // one read that one again
    for (int r0 = 0; r0 < live; r0 += 8) {
      Raw8<KV> u[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) u[r] = load8<KV>(p.k_cache, (row0 + min(r0 + r, live - 1)) * p.D + c * 8);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        uint32_t w[4];
        pairs8<KV>(u[r], w);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool first = r0 + r == 0;
          lo[k] = first ? w[k] : pair_extreme<KV == kBF16c, false>(lo[k], w[k]);
          hi[k] = first ? w[k] : pair_extreme<KV == kBF16c, true>(hi[k], w[k]);
        }
      }
    }
    const int64_t at = (static_cast<int64_t>(b) * p.Hkv + h) * 2 * p.D + c * 8;
    store8<KV>(p.bounds, at, lo);
    store8<KV>(p.bounds, at + p.D, hi);
  }
}

// ---- scores -----------------------------------------------------------------
// The bound max over heads g of  sum_d max(q, 0) hi + min(q, 0) lo  is a matrix
// product: the block's 2 D bounds (low, then high) times the head's (min(q, 0),
// max(q, 0)).  Each bound is read once (2 D elements per block and kv head,
// 4 D G operations), so the read is the floor.  A warp takes 16 blocks of one
// (sequence, kv head) as the 16 rows of m16n8k16 MMAs and up to 16 query heads
// as columns.  The order of the inner dimension is free, so a lane's 16-byte
// load is its A fragment as it stands: lane (r, c) = (lane / 4, lane % 4)
// takes the c-th 16 bytes of each 64-byte segment of rows r and r + 8, which
// makes whole-sector reads and needs no shared memory; the query fragments
// take the same channels and stay in registers over the warp's tiles.
//
// A lane reads back only the pieces it copied itself, so a warp's tile goes
// through shared memory by asynchronous 16-byte copies with no barrier: the
// copies in flight (8 KB per warp) do not cost registers, and many warps per SM
// hide one another's waits.  Measured over 8 contexts of 32K to 128K tokens
// (189 MB): rings of 3, 2, 1 tiles per warp 46, 40, 34 us (fewer tiles, more
// warps), 0.82 of a plain copy's rate; kv heads of the same blocks far apart in
// the grid 7 us more (512-byte pieces of memory, 4 KB with their neighbours).
//
// E4M3 bounds are widened to f16 (exact); bf16 queries are then scaled per
// head by a power of two into f16's range (exact but for entries below 2^-29
// of the head's largest), which the score is divided by.
constexpr int kScoreWarps = 4;
constexpr int kScoreTile = 16;  // blocks per warp tile

template <int KV, int D>
struct ScoreGeom {
  static constexpr bool E4 = KV == kE4M3c;
  static constexpr int EPL = E4 ? 16 : 8;       // elements per 16-byte piece
  static constexpr int SEGS = D / (4 * EPL);    // 64-byte segments per half
  static constexpr int STEPS = EPL / 4;         // MMA k-steps per segment
  static constexpr int PIECES = 4 * SEGS;       // 16-byte pieces of a lane per tile: side, segment, row
  static constexpr int TILE_BYTES = PIECES * 32 * 16;
  static constexpr int GROUP = 8192 / TILE_BYTES;  // tiles fetched at once: 8 KB per warp
  static constexpr int SMEM = kScoreWarps * GROUP * TILE_BYTES;
};

template <int KV, int D, int NT>
__global__ void __launch_bounds__(kScoreWarps * 32) block_scores_kernel(const ScoresParams p, int chunks,
                                                                        int tiles_per_warp) {
  using Gm = ScoreGeom<KV, D>;
  constexpr bool E4 = Gm::E4;
  constexpr int EPL = Gm::EPL, SEGS = Gm::SEGS, STEPS = Gm::STEPS, GROUP = Gm::GROUP;
  extern __shared__ __align__(16) uint8_t tiles[];
  pdl_enter();
  constexpr bool B0 = KV == kBF16c;      // operands in bf16, else f16
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
  // neighbouring CTAs take the kv heads of the same blocks, whose bounds are
  // neighbours in memory
  const int h = blockIdx.x % p.Hkv, sc = blockIdx.x / p.Hkv;
  const int chunk = sc % chunks, s = sc / chunks, sh = s * p.Hkv + h;
  const int L = clamped_length(p.context_lens, s, p.maxB * p.bs, p.err);
  const int nb = (L + p.bs - 1) / p.bs;
  const int tile0 = chunk * kScoreWarps * tiles_per_warp + warp;
  const int32_t* table = p.block_tables + static_cast<int64_t>(s) * p.maxB;
  float* out = p.scores + static_cast<int64_t>(sh) * p.maxB;
  const uint32_t mine = smem_u32(tiles) + (warp * GROUP * Gm::PIECES * 32 + lane) * 16;  // piece i: + 512 i

  // the lane's two table entries of tile t, -1 past the context
  auto ids_of = [&](int t, int (&b)[2]) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int j = (tile0 + t * kScoreWarps) * kScoreTile + r + 8 * e;
      b[e] = t < tiles_per_warp && j < nb ? load_written(table + j) : -1;
      if (t < tiles_per_warp && j < nb && (b[e] < 0 || b[e] >= p.num_blocks) && c == 0)
        atomicOr(p.err, PA_DEVERR_BLOCK_ID);
    }
  };
  auto fetch = [&](uint32_t dst, const int (&b)[2]) {  // a row past the context or outside the pool: zeros
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const bool on = b[e] >= 0 && b[e] < p.num_blocks;
      const uint8_t* src = static_cast<const uint8_t*>(p.bounds) +
                           (static_cast<int64_t>(on ? b[e] : 0) * p.Hkv + h) * (2 * D * (E4 ? 1 : 2)) + 16 * c;
#pragma unroll
      for (int i = 0; i < 2 * SEGS; ++i) copy16_async_or_zero(dst + (2 * i + e) * 512, src + 64 * i, on);
    }
  };

  for (int g0 = 0; g0 < p.G; g0 += 8 * NT) {
    // query fragments: low and high side of the lane's channels of head g0 + 8 nt + r
    uint32_t qf[NT][2][SEGS][STEPS][2];
    float inv[NT][2];  // power of two each of the lane's two columns was scaled by, inverted
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int g = g0 + 8 * nt + r;
      uint32_t raw[SEGS][STEPS][2];
      const uint16_t* q = static_cast<const uint16_t*>(p.q) + (static_cast<int64_t>(s) * p.Hq + h * p.G + g) * D;
#pragma unroll
      for (int i = 0; i < SEGS; ++i)
#pragma unroll
        for (int k = 0; k < STEPS; k += 2) {
          const uint4 u = g < p.G ? load_written(reinterpret_cast<const uint4*>(q + (4 * i + c) * EPL + 4 * k))
                                  : make_uint4(0u, 0u, 0u, 0u);
          raw[i][k][0] = u.x;
          raw[i][k][1] = u.y;
          raw[i][k + 1][0] = u.z;
          raw[i][k + 1][1] = u.w;
        }
      inv[nt][0] = inv[nt][1] = 1.f;
      if (E4 && p.q_bf16) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < SEGS; ++i)
#pragma unroll
          for (int k = 0; k < STEPS; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float a = fabsf(__uint_as_float(raw[i][k][e] << 16));
              const float b = fabsf(__uint_as_float(raw[i][k][e] & 0xFFFF0000u));
              if (a < CUDART_INF_F) m = fmaxf(m, a);
              if (b < CUDART_INF_F) m = fmaxf(m, b);
            }
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        int ex = 15;
        if (m > 0.f) frexpf(m, &ex);  // m = f 2^ex, f in [0.5, 1)
        const int e2 = min(15 - ex, 126);
        const float mul = ldexpf(1.f, e2);
#pragma unroll
        for (int i = 0; i < SEGS; ++i)
#pragma unroll
          for (int k = 0; k < STEPS; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const __half2 v = __floats2half2_rn(__uint_as_float(raw[i][k][e] << 16) * mul,
                                                  __uint_as_float(raw[i][k][e] & 0xFFFF0000u) * mul);
              raw[i][k][e] = *reinterpret_cast<const uint32_t*>(&v);
            }
        const float back = ldexpf(1.f, -e2);  // of head r; the accumulators hold heads 2 c and 2 c + 1
        inv[nt][0] = __shfl_sync(0xFFFFFFFFu, back, 8 * c);
        inv[nt][1] = __shfl_sync(0xFFFFFFFFu, back, 8 * c + 4);
      }
#pragma unroll
      for (int i = 0; i < SEGS; ++i)
#pragma unroll
        for (int k = 0; k < STEPS; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            qf[nt][0][i][k][e] = pair_extreme<B0, false>(raw[i][k][e], 0u);
            qf[nt][1][i][k][e] = pair_extreme<B0, true>(raw[i][k][e], 0u);
          }
    }

    int ids[GROUP][2];
#pragma unroll
    for (int i = 0; i < GROUP; ++i) ids_of(i, ids[i]);
    for (int t = 0; t < tiles_per_warp; ++t) {
      const int j0 = (tile0 + t * kScoreWarps) * kScoreTile;
      if (j0 >= p.maxB) break;
      if (t % GROUP == 0) {
#pragma unroll
        for (int i = 0; i < GROUP; ++i) fetch(mine + i * Gm::PIECES * 512, ids[i]);
        copies_commit();
#pragma unroll
        for (int i = 0; i < GROUP; ++i) ids_of(t + GROUP + i, ids[i]);
        copies_wait<0>();
      }
      const uint32_t tile = mine + t % GROUP * Gm::PIECES * 512;
      float acc[NT][2][4];  // the low and the high side's sums
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
      if (j0 < nb) {
#pragma unroll
        for (int i = 0; i < SEGS; ++i)
#pragma unroll
          for (int side = 0; side < 2; ++side) {
            uint32_t wx[4], wy[4];
            load16_shared(tile + 2 * (side * SEGS + i) * 512, wx);
            load16_shared(tile + (2 * (side * SEGS + i) + 1) * 512, wy);
#pragma unroll
            for (int k = 0; k < STEPS; ++k) {
              uint32_t a[4];
              if constexpr (E4) {
                e4m3x4_to_f16x2x2(wx[k], a[0], a[2]);
                e4m3x4_to_f16x2x2(wy[k], a[1], a[3]);
              } else {
                a[0] = wx[2 * k];
                a[2] = wx[2 * k + 1];
                a[1] = wy[2 * k];
                a[3] = wy[2 * k + 1];
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816<KV == kBF16c>(acc[nt][side], a, qf[nt][side][i][k][0], qf[nt][side][i][k][1]);
            }
          }
      }
      float best[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (g0 + 8 * nt + 2 * c + i < p.G)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              best[e] = max_nan(best[e], (acc[nt][0][2 * e + i] + acc[nt][1][2 * e + i]) * inv[nt][i]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        best[e] = max_nan(best[e], __shfl_xor_sync(0xFFFFFFFFu, best[e], 1));
        best[e] = max_nan(best[e], __shfl_xor_sync(0xFFFFFFFFu, best[e], 2));
        const int j = j0 + r + 8 * e;
        if (c == 0 && j < p.maxB) {
          // wider groups: the maximum so far is this lane's own earlier write
          if (g0 > 0) best[e] = max_nan(best[e], out[j]);
          out[j] = j < nb ? best[e] : -CUDART_INF_F;
        }
      }
    }
  }
}

// ---- selection --------------------------------------------------------------
// One CTA per (sequence, kv head): a row of scores is a few dozen KB, so the
// selection is bound by the latency and the instructions of its steps.
//  - The scores are read once, as unsigned keys of the same order (the first
//    and the last blocks of the context get the largest key), into registers,
//    16 per thread; rows of more blocks go to shared memory, and beyond that are
//    read again from memory.  The least and largest competing keys are found.
//  - A histogram of up to 2048 equal bins over that range gives the bin in which the
//    count of blocks to take runs out (scores of one query lie close together:
//    bins by their leading bits would hold nearly all of them).
//  - If that bin holds few keys they are gathered, each counts those above it,
//    and the one whose place is the last to be taken is the last key.  If it
//    holds many, the next histogram spans their own range, until they are few
//    or all equal.
//  - Ballots mark the blocks taken, 32 consecutive ones at a time; a scan of
//    their counts gives the places, and each lane writes the ids of one ballot
//    in context order.  Of the blocks with the last key the lowest indexes are
//    taken.
// (256 of up to 8192 blocks for 32 sequences x 8 heads: 30.7 us with four
// passes of leading-digit histograms over the scores in memory, 15.5 with the
// steps above over shared memory, 11.9 over registers.)
constexpr int kSelectPerThread = 16;         // keys in registers
constexpr int kSelectSmemKeys = 50 * 1024;   // more blocks than this are read again from memory
constexpr uint32_t kForcedKey = 0xFFFFFFFFu;
enum : int { kKeysInRegs = 0, kKeysInSmem = 1, kKeysInMemory = 2 };

__device__ __forceinline__ uint32_t score_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 and 0 are equal
  const uint32_t k = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
  return x != x ? kForcedKey - 1 : k;  // NaN before every number
}

// Exclusive sum of the warps' counts `v` (the same in all lanes) over the warps
// before this one, and the total; `sums` holds a word per warp.
__device__ __forceinline__ uint32_t warps_scan(uint32_t v, uint32_t* sums, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  if (lane == 0) sums[warp] = v;
  __syncthreads();
  const uint32_t u = lane < nw ? sums[lane] : 0;
  total = __reduce_add_sync(0xFFFFFFFFu, u);
  const uint32_t before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? u : 0);
  __syncthreads();  // sums may be reused
  return before;
}

__device__ __forceinline__ uint32_t lanes_before(uint32_t v) {  // exclusive sum over the lanes
  const int lane = threadIdx.x & 31;
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += u;
  }
  return incl - v;
}

template <int WHERE, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) select_blocks_kernel(const SelectParams p) {
  constexpr int K = kSelectPerThread, NW = NT / 32;
  constexpr int BINS = NT < 512 ? 4 * NT : 2048, LOG_BINS = NT == 64 ? 8 : (NT == 128 ? 9 : (NT == 256 ? 10 : 11));
  constexpr int FEW = NT < 128 ? NT : 128;  // a thread each
  extern __shared__ uint32_t keys[];
  __shared__ int hist[BINS];
  __shared__ uint32_t sums[WHERE == kKeysInRegs ? K * NW : 32];
  __shared__ uint32_t few[FEW];
  __shared__ uint32_t sh_lo, sh_hi;
  __shared__ int sh_need, sh_count, sh_bin, sh_few, sh_last;
  pdl_enter();
  const int s = blockIdx.x / p.Hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int L = clamped_length(p.context_lens, s, p.maxB * p.bs, p.err);
  const int nb = (L + p.bs - 1) / p.bs;
  const float* score = p.scores + static_cast<int64_t>(blockIdx.x) * p.maxB;
  const int32_t* table = p.block_tables + static_cast<int64_t>(s) * p.maxB;
  int32_t* out = p.tables + static_cast<int64_t>(blockIdx.x) * p.n;
  const int sink = min(p.sink, nb), recent0 = max(nb - p.recent, sink);  // [sink, recent0) compete
  const bool all = nb <= p.n;
  const int total = min(nb, p.n);
  int need = total - (sink + nb - recent0);  // taken by score
  const auto read_key = [&](int j) {
    return all || j < sink || j >= recent0 ? kForcedKey : score_key(load_written(score + j));
  };
  // registers: block i NT + tid is the thread's i-th, 0 past the context (no score's key is)
  uint32_t mine[K];
  if constexpr (WHERE == kKeysInRegs) {
    float x[K];  // all loads before the first is looked at
#pragma unroll
    for (int i = 0; i < K; ++i) x[i] = !all && i * NT + tid < nb ? load_written(score + i * NT + tid) : 0.f;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int j = i * NT + tid;
      mine[i] = all || j < sink || j >= recent0 ? kForcedKey : score_key(x[i]);
      if (j >= nb) mine[i] = 0;
    }
  }
  const auto key = [&](int j) { return WHERE == kKeysInSmem ? keys[j] : read_key(j); };
  // work(key) for each of the thread's keys
  const auto each = [&](auto work) {
    if constexpr (WHERE == kKeysInRegs) {
#pragma unroll
      for (int i = 0; i < K; i += 4)
        if (i * NT < nb) {
          work(mine[i]);
          work(mine[i + 1]);
          work(mine[i + 2]);
          work(mine[i + 3]);
        }
    } else {
#pragma unroll 4
      for (int j = tid; j < nb; j += NT) work(key(j));
    }
  };
  uint32_t last_key = kForcedKey - 1;  // blocks with larger keys are taken, and
  int equal_taken = 0;                 // the first so many with this one
  if (tid == 0) {
    sh_lo = kForcedKey;
    sh_hi = 0;
    sh_last = 0;
  }
  __syncthreads();
  if (!all) {
    uint32_t lo = kForcedKey, hi = 0;
    const auto widen = [&](uint32_t k) {
      if (k - 1 < kForcedKey - 1) {  // neither forced nor past the context
        lo = min(lo, k);
        hi = max(hi, k);
      }
    };
    if constexpr (WHERE == kKeysInSmem) {
#pragma unroll 8
      for (int j = tid; j < nb; j += NT) {
        const uint32_t k = read_key(j);
        keys[j] = k;
        widen(k);
      }
    } else {
      each(widen);
    }
    const auto share_range = [&]() {  // least and largest over the CTA (sh_lo, sh_hi reset before)
      lo = __reduce_min_sync(0xFFFFFFFFu, lo);
      hi = __reduce_max_sync(0xFFFFFFFFu, hi);
      if (lane == 0) {
        atomicMin(&sh_lo, lo);
        atomicMax(&sh_hi, hi);
      }
      __syncthreads();
      lo = sh_lo;
      hi = sh_hi;
    };
    share_range();
    int count = recent0 - sink;  // keys in [lo, hi], of which `need` are taken
    while (need > 0) {
      if (lo == hi || need == count) {
        // all equal, or all taken (above lo - 1: no key is 0, -infinity's is the least)
        last_key = need == count ? lo - 1 : lo;
        equal_taken = need == count ? 0 : need;
        break;
      }
      const uint32_t span = hi - lo;
      const int shift = max(32 - LOG_BINS - __clz(span), 0);  // span >> shift < BINS
      for (int i = tid; i < BINS; i += NT) hist[i] = 0;
      if (tid == 0) sh_few = 0;
      __syncthreads();
      each([&](uint32_t k) {
        if (k - lo <= span) atomicAdd(&hist[(k - lo) >> shift], 1);
      });
      __syncthreads();
      // bins from the highest: the one in which `need` runs out
      constexpr int per = BINS / NT;
      const int top = BINS - 1 - tid * per;
      uint32_t held = 0, sum;
#pragma unroll
      for (int i = 0; i < per; ++i) held += hist[top - i];
      const uint32_t within = lanes_before(held);
      int before = warps_scan(__shfl_sync(0xFFFFFFFFu, within + held, 31), sums, sum) + within;
      if (before < need && need <= before + static_cast<int>(held)) {
        for (int i = 0; i < per; ++i) {
          const int c = hist[top - i];
          if (need <= before + c) {
            sh_need = need - before;
            sh_count = c;
            sh_bin = top - i;
            break;
          }
          before += c;
        }
      }
      if (tid == 0) {
        sh_lo = kForcedKey;
        sh_hi = 0;
      }
      __syncthreads();
      need = sh_need;
      count = sh_count;
      // the bin's keys, at most the range's largest
      const uint32_t bin_lo = lo + (static_cast<uint32_t>(sh_bin) << shift);
      const uint32_t bin_top = min((1u << shift) - 1u, hi - bin_lo);
      if (count <= FEW) {
        each([&](uint32_t k) {
          if (k - bin_lo <= bin_top) few[atomicAdd(&sh_few, 1)] = k;
        });
        __syncthreads();
        if (tid < count) {
          const uint32_t k = few[tid];
          int above = 0, equal = 0;
          for (int i = 0; i < count; ++i) {
            above += few[i] > k;
            equal += few[i] == k;
          }
          if (above < need && need <= above + equal) {  // the same for all of this key
            sh_lo = k;
            sh_count = need - above;
          }
        }
        __syncthreads();
        last_key = sh_lo;
        equal_taken = sh_count;
        break;
      }
      lo = kForcedKey;
      hi = 0;
      each([&](uint32_t k) {
        if (k - bin_lo <= bin_top) {
          lo = min(lo, k);
          hi = max(hi, k);
        }
      });
      share_range();
    }
  }
  // Writes the blocks that `sure` and `equal` mark from block `first` on;
  // `before`: the sure blocks before them (low half) and those of the last key (high half).
  int taken = 0, equals = 0;  // in memory: blocks taken and blocks of the last key in earlier passes
  const auto write = [&](uint32_t sure, uint32_t equal, int first, uint32_t before) {
    int e_rank = equals + static_cast<int>(before >> 16);
    // places: the sure blocks before, and those of the last key before, as far as they are taken
    int at = taken + static_cast<int>(before & 0xFFFFu) + min(e_rank, equal_taken) - min(equals, equal_taken);
    for (uint32_t m = sure | equal; m; m &= m - 1) {
      const int i = __ffs(m) - 1;
      const bool is_equal = equal >> i & 1;
      if (!is_equal || e_rank < equal_taken) {
        out[at++] = load_written(table + first + i);
        if (first + i == nb - 1) sh_last = 1;
      }
      e_rank += is_equal;
    }
  };
  // counts in 16 bits each: at most 32 x 1024 blocks a pass
  const auto counts = [](uint32_t sure, uint32_t equal) -> uint32_t { return __popc(sure) | __popc(equal) << 16; };
  if constexpr (WHERE == kKeysInRegs) {
    uint32_t sure = 0, equal = 0;  // lane i: the ballots of the warp's i-th blocks
#pragma unroll
    for (int i = 0; i < K; ++i) {
      if (i * NT >= nb) break;
      const uint32_t sm = __ballot_sync(0xFFFFFFFFu, mine[i] > last_key);
      const uint32_t em = __ballot_sync(0xFFFFFFFFu, mine[i] == last_key);
      if (lane == i) {
        sure = sm;
        equal = em;
      }
    }
    // exclusive sums in block order (i, then warp) by the first warp
    if (lane < K) sums[lane * NW + warp] = counts(sure, equal);
    __syncthreads();
    if (warp == 0) {
      constexpr int per = K * NW / 32;
      uint32_t v[per], held = 0;
#pragma unroll
      for (int i = 0; i < per; ++i) {
        v[i] = sums[lane * per + i];
        held += v[i];
      }
      uint32_t before = lanes_before(held);
#pragma unroll
      for (int i = 0; i < per; ++i) {
        sums[lane * per + i] = before;
        before += v[i];
      }
    }
    __syncthreads();
    if (lane < K) write(sure, equal, lane * NT + warp * 32, sums[lane * NW + warp]);
  } else {
    // each warp looks at `steps` (at most 32) times 32 consecutive blocks and
    // keeps step i's ballots in lane i
    const int steps = min((nb + NT - 1) / NT, 32);
    for (int base = 0; base < nb; base += steps * NT) {
      const int first = base + warp * steps * 32;
      uint32_t sure = 0, equal = 0;
      for (int i = 0; i < steps; ++i) {
        const int j = first + 32 * i + lane;
        const uint32_t k = j < nb ? (all ? kForcedKey : key(j)) : 0;
        const uint32_t sm = __ballot_sync(0xFFFFFFFFu, k > last_key);
        const uint32_t em = __ballot_sync(0xFFFFFFFFu, k == last_key);
        if (lane == i) {
          sure = sm;
          equal = em;
        }
      }
      const uint32_t held = counts(sure, equal), within = lanes_before(held);
      uint32_t sum;
      const uint32_t before = warps_scan(__shfl_sync(0xFFFFFFFFu, within + held, 31), sums, sum) + within;
      write(sure, equal, first + 32 * lane, before);
      const int e_all = static_cast<int>(sum >> 16);
      taken += static_cast<int>(sum & 0xFFFFu) + min(equals + e_all, equal_taken) - min(equals, equal_taken);
      equals += e_all;
    }
  }
  for (int i = total + tid; i < p.n; i += NT) out[i] = -1;
  __syncthreads();
  if (tid == 0) p.lens[blockIdx.x] = total * p.bs - (sh_last ? nb * p.bs - L : 0);
}

}  // namespace

cudaError_t launch_block_bounds(const BoundsParams& p, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(p.S) * static_cast<unsigned>(p.touched);
  auto kern = p.kv_dtype == PA_F16    ? block_bounds_kernel<kF16c>
              : p.kv_dtype == PA_BF16 ? block_bounds_kernel<kBF16c>
                                      : block_bounds_kernel<kE4M3c>;
  return launch_in_order(kern, grid, 128, 0, st, p);
}

template <int KV, int D, int NT>
static cudaError_t launch_scores_nt(const ScoresParams& p, cudaStream_t st) {
  const int tiles = (p.maxB + kScoreTile - 1) / kScoreTile;
  const int64_t heads = static_cast<int64_t>(p.S) * p.Hkv;
  // two groups of tiles share a warp's query fragments once there are warps enough
  // (8 tiles of 8 KB per warp: 36 us at the size above, 4: 35, 2: 34)
  constexpr int kGroup = ScoreGeom<KV, D>::GROUP;
  const int tpw =
      heads * tiles >= int64_t(p.sms) * 32 * kGroup ? 2 * kGroup : (heads * tiles >= int64_t(p.sms) * 16 ? kGroup : 1);
  const int chunks = (tiles + kScoreWarps * tpw - 1) / (kScoreWarps * tpw);
  auto kern = block_scores_kernel<KV, D, NT>;
  const int smem = ScoreGeom<KV, D>::SMEM;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_in_order(kern, static_cast<unsigned>(heads * chunks), kScoreWarps * 32, smem, st, p, chunks, tpw);
}

template <int KV, int D>
static cudaError_t launch_scores(const ScoresParams& p, cudaStream_t st) {
  return p.G <= 8 ? launch_scores_nt<KV, D, 1>(p, st) : launch_scores_nt<KV, D, 2>(p, st);
}

cudaError_t launch_block_scores(const ScoresParams& p, cudaStream_t st) {
  if (p.kv_dtype == PA_F16) return p.D == 64 ? launch_scores<kF16c, 64>(p, st) : launch_scores<kF16c, 128>(p, st);
  if (p.kv_dtype == PA_BF16) return p.D == 64 ? launch_scores<kBF16c, 64>(p, st) : launch_scores<kBF16c, 128>(p, st);
  return p.D == 64 ? launch_scores<kE4M3c, 64>(p, st) : launch_scores<kE4M3c, 128>(p, st);
}

cudaError_t launch_select_blocks(const SelectParams& p, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(p.S) * p.Hkv);
  // registers where 16 keys per thread hold the row.  Many rows: as few threads
  // as hold a row, so that barriers are cheap and more rows share an SM (2048
  // rows of 256 blocks 10.0, 12.9, 20.8, 38.5 us with 64, 128, 256, 512 threads; of 1024
  // blocks 11.8, 15.4, 21.9, 37.2).  Few: each row's own steps count (256 rows of 256
  // blocks 6.0, 5.5, 5.5, 7.0; 8 rows of 2048: 5.6, 5.2, 5.1 with 128, 256, 512).
  constexpr int K = kSelectPerThread;
  const bool alone = grid <= static_cast<unsigned>(p.sms), many = grid > 4 * static_cast<unsigned>(p.sms);
  auto kern = select_blocks_kernel<kKeysInMemory, 512>;
  int threads = 512, smem = 0;
  if (p.maxB <= K * 64 && many) {
    kern = select_blocks_kernel<kKeysInRegs, 64>;
    threads = 64;
  } else if (p.maxB <= K * 128 && !alone) {
    kern = select_blocks_kernel<kKeysInRegs, 128>;
    threads = 128;
  } else if (p.maxB <= K * 256 && (!alone || p.maxB <= 2048)) {
    kern = select_blocks_kernel<kKeysInRegs, 256>;
    threads = 256;
  } else if (p.maxB <= K * 512 && (!alone || p.maxB <= 4096)) {
    kern = select_blocks_kernel<kKeysInRegs, 512>;
  } else if (p.maxB <= K * 1024) {
    kern = select_blocks_kernel<kKeysInRegs, 1024>;
    threads = 1024;
  } else if (p.maxB <= kSelectSmemKeys) {
    kern = select_blocks_kernel<kKeysInSmem, 1024>;
    threads = 1024;
    smem = p.maxB * 4;
  }
  if (smem > 0) {
    // the kernel's limit, the same in every call: another thread may set it
    // between this and the launch
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelectSmemKeys * 4);
    if (e != cudaSuccess) return e;
  }
  return launch_in_order(kern, grid, threads, smem, st, p);
}

}  // namespace pa
