// Choosing the blocks a decode step attends to: the bounds of each block's
// keys, their scores against the step's queries, and the selection.
#include <math_constants.h>

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
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Eight cache values at element index `at` (a multiple of 8), widened exactly.
template <int KV>
__device__ __forceinline__ void load8(const void* base, int64_t at, float (&x)[8]) {
  if constexpr (KV == kE4M3c) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(base) + at));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = i < 2 ? u.x : u.y;
      const float2 v = __half22float2(
          __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * (i & 1))), __NV_E4M3)));
      x[2 * i] = v.x;
      x[2 * i + 1] = v.y;
    }
  } else {
    widen8<KV == kBF16c>(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at)), x);
  }
}

template <int KV>
__device__ __forceinline__ void store8(void* base, int64_t at, const float (&x)[8]) {
  if constexpr (KV == kE4M3c)
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + at) = quantise8(x, 1.f);  // exact: the values are codes
  else
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = narrow8<KV == kBF16c>(x);
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
// kv head reads the block's live keys and keeps their least and largest.
template <int KV>
__global__ void __launch_bounds__(128) block_bounds_kernel(const BoundsParams p) {
  const int s = blockIdx.y;
  const int L = clamped_length(p.context_lens, s, p.maxB * p.bs, p.err);
  const int j = max(L - p.num_new, 0) / p.bs + blockIdx.x;
  const int live = min(p.bs, L - j * p.bs);
  if (live <= 0) return;
  const int b = __ldg(p.block_tables + static_cast<int64_t>(s) * p.maxB + j);
  if (b < 0 || b >= p.num_blocks) {
    if (threadIdx.x == 0) atomicOr(p.err, PA_DEVERR_BLOCK_ID);
    return;
  }
  const int pieces = p.D / 8;
  for (int i = threadIdx.x; i < p.Hkv * pieces; i += blockDim.x) {
    const int h = i / pieces, c = i % pieces;
    const int64_t row0 = (static_cast<int64_t>(b) * p.Hkv + h) * p.bs;
    float lo[8], hi[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      lo[k] = CUDART_INF_F;
      hi[k] = -CUDART_INF_F;
    }
#pragma unroll 8
    for (int r = 0; r < live; ++r) {
      float x[8];
      load8<KV>(p.k_cache, (row0 + r) * p.D + c * 8, x);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        lo[k] = min_nan(lo[k], x[k]);
        hi[k] = max_nan(hi[k], x[k]);
      }
    }
    const int64_t at = (static_cast<int64_t>(b) * p.Hkv + h) * 2 * p.D + c * 8;
    store8<KV>(p.bounds, at, lo);
    store8<KV>(p.bounds, at + p.D, hi);
  }
}

// ---- scores -----------------------------------------------------------------
// A warp per (sequence, kv head, block): the block's low and high halves are
// spread over the lanes, and each query head's sum is a shuffle reduction.
constexpr int kScoreWarps = 8, kScoreBlocksPerWarp = 8;

template <int KV, int D>
__global__ void __launch_bounds__(kScoreWarps * 32) block_scores_kernel(const ScoresParams p) {
  __shared__ __align__(16) uint16_t q_sh[128 * D];
  const int s = blockIdx.z, h = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int L = clamped_length(p.context_lens, s, p.maxB * p.bs, p.err);
  const int nb = (L + p.bs - 1) / p.bs;
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                  (static_cast<int64_t>(s) * p.Hq + h * p.G) * D);
  for (int i = threadIdx.x; i < p.G * D / 8; i += blockDim.x) reinterpret_cast<uint4*>(q_sh)[i] = __ldg(q + i);
  __syncthreads();
  constexpr int PIECES = D / 8;  // lanes per half
  const bool high = (lane / PIECES) & 1, on = lane < 2 * PIECES;
  const int c = lane % PIECES;
  float* out = p.scores + (static_cast<int64_t>(s) * p.Hkv + h) * p.maxB;
  for (int k = 0; k < kScoreBlocksPerWarp; ++k) {
    const int j = (blockIdx.x * kScoreBlocksPerWarp + k) * kScoreWarps + warp;
    if (j >= p.maxB) break;
    if (j >= nb) {
      if (lane == 0) out[j] = -CUDART_INF_F;
      continue;
    }
    const int b = __ldg(p.block_tables + static_cast<int64_t>(s) * p.maxB + j);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (b < 0 || b >= p.num_blocks) {  // bounds of zeros
      if (lane == 0) atomicOr(p.err, PA_DEVERR_BLOCK_ID);
    } else if (on) {
      load8<KV>(p.bounds, ((static_cast<int64_t>(b) * p.Hkv + h) * 2 + high) * D + c * 8, x);
    }
    float best = -CUDART_INF_F;
    for (int g = 0; g < p.G; ++g) {
      float qv[8], sum = 0.f;
      const uint4 u = *reinterpret_cast<const uint4*>(q_sh + g * D + c * 8);
      if (p.q_bf16)
        widen8<true>(u, qv);
      else
        widen8<false>(u, qv);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(high ? max_nan(qv[i], 0.f) : min_nan(qv[i], 0.f), x[i], sum);
      if (!on) sum = 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      best = max_nan(best, sum);
    }
    if (lane == 0) out[j] = best;
  }
}

// ---- selection --------------------------------------------------------------
// One CTA per (sequence, kv head).  Scores map to unsigned keys of the same
// order; four passes of 256-bin histograms find the key of the last block
// taken and how many of equal key are taken; a pass in index order writes the
// blocks, lowest index first.
constexpr int kSelectThreads = 512;

__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0xFFFFFFFFu;  // NaN before everything
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 and 0 are equal
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelectThreads) select_blocks_kernel(const SelectParams p) {
  __shared__ int hist[256];
  __shared__ int warp_sum[kSelectThreads / 32][2];
  __shared__ uint32_t sh_prefix;
  __shared__ int sh_need, sh_last;
  const int s = blockIdx.x / p.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int L = clamped_length(p.context_lens, s, p.maxB * p.bs, p.err);
  const int nb = (L + p.bs - 1) / p.bs;
  const float* score = p.scores + static_cast<int64_t>(blockIdx.x) * p.maxB;
  const int32_t* table = p.block_tables + static_cast<int64_t>(s) * p.maxB;
  int32_t* out = p.tables + static_cast<int64_t>(blockIdx.x) * p.n;
  const int sink = min(p.sink, nb), recent0 = max(nb - p.recent, sink);  // [sink, recent0) compete
  const bool all = nb <= p.n;
  const int total = min(nb, p.n);
  int need = total - (sink + nb - recent0);  // taken by score
  uint32_t last_key = 0;                     // key of the last block taken
  int equal_taken = 0;                       // blocks of that key taken
  if (!all && need > 0) {
    uint32_t prefix = 0, mask = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelectThreads) hist[i] = 0;
      __syncthreads();
      for (int j = sink + tid; j < recent0; j += kSelectThreads) {
        const uint32_t k = score_key(__ldg(score + j));
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (warp == 0) {  // the bin, from the highest, in which `need` runs out
        int c[8], mine = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          c[i] = hist[255 - (lane * 8 + i)];
          mine += c[i];
        }
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
          if (lane >= o) incl += v;
        }
        int before = incl - mine;
        if (before < need && need <= incl) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (before < need && need <= before + c[i]) {
              sh_prefix = prefix | (static_cast<uint32_t>(255 - (lane * 8 + i)) << shift);
              sh_need = need - before;
            }
            before += c[i];
          }
        }
      }
      __syncthreads();
      prefix = sh_prefix;
      need = sh_need;
      mask |= 255u << shift;
    }
    last_key = prefix;
    equal_taken = need;
  }
  // in index order: blocks before, and blocks of the last key before
  if (tid == 0) sh_last = 0;
  int taken = 0, equals = 0;
  for (int j0 = 0; j0 < nb; j0 += kSelectThreads) {
    const int j = j0 + tid;
    bool sure = false, equal = false;
    if (j < nb) {
      sure = all || j < sink || j >= recent0;
      if (!sure && equal_taken > 0) {
        const uint32_t k = score_key(__ldg(score + j));
        sure = k > last_key;
        equal = k == last_key;
      }
    }
    const unsigned em = __ballot_sync(0xFFFFFFFFu, equal);
    const unsigned sm = __ballot_sync(0xFFFFFFFFu, sure);
    if (lane == 0) {
      warp_sum[warp][0] = __popc(sm);
      warp_sum[warp][1] = __popc(em);
    }
    __syncthreads();
    int s_before = 0, e_before = 0, s_all = 0, e_all = 0;
    for (int w = 0; w < kSelectThreads / 32; ++w) {
      const int a = warp_sum[w][0], b = warp_sum[w][1];
      if (w < warp) {
        s_before += a;
        e_before += b;
      }
      s_all += a;
      e_all += b;
    }
    const unsigned below = (1u << lane) - 1u;
    // blocks of the last key before this one; the first equal_taken are taken
    const int e_rank = equals + e_before + __popc(em & below);
    const bool take = sure || (equal && e_rank < equal_taken);
    const int at = taken + s_before + __popc(sm & below) + min(e_rank, equal_taken) - min(equals, equal_taken);
    if (take) {
      out[at] = __ldg(table + j);
      if (j == nb - 1) sh_last = 1;
    }
    taken += s_all + min(equals + e_all, equal_taken) - min(equals, equal_taken);
    equals += e_all;
    __syncthreads();
  }
  for (int i = total + tid; i < p.n; i += kSelectThreads) out[i] = -1;
  __syncthreads();
  if (tid == 0) p.lens[blockIdx.x] = total * p.bs - (sh_last ? nb * p.bs - L : 0);
}

}  // namespace

cudaError_t launch_block_bounds(const BoundsParams& p, cudaStream_t st) {
  const int touched = (p.num_new + p.bs - 2) / p.bs + 1;
  const dim3 grid(static_cast<unsigned>(min(touched, p.maxB)), static_cast<unsigned>(p.S));
  if (p.kv_dtype == PA_F16)
    block_bounds_kernel<kF16c><<<grid, 128, 0, st>>>(p);
  else if (p.kv_dtype == PA_BF16)
    block_bounds_kernel<kBF16c><<<grid, 128, 0, st>>>(p);
  else
    block_bounds_kernel<kE4M3c><<<grid, 128, 0, st>>>(p);
  return cudaGetLastError();
}

template <int KV>
static void launch_scores(const ScoresParams& p, cudaStream_t st) {
  const int per = kScoreWarps * kScoreBlocksPerWarp;
  const dim3 grid(static_cast<unsigned>((p.maxB + per - 1) / per), static_cast<unsigned>(p.Hkv),
                  static_cast<unsigned>(p.S));
  if (p.D == 64)
    block_scores_kernel<KV, 64><<<grid, kScoreWarps * 32, 0, st>>>(p);
  else
    block_scores_kernel<KV, 128><<<grid, kScoreWarps * 32, 0, st>>>(p);
}

cudaError_t launch_block_scores(const ScoresParams& p, cudaStream_t st) {
  if (p.kv_dtype == PA_F16)
    launch_scores<kF16c>(p, st);
  else if (p.kv_dtype == PA_BF16)
    launch_scores<kBF16c>(p, st);
  else
    launch_scores<kE4M3c>(p, st);
  return cudaGetLastError();
}

cudaError_t launch_select_blocks(const SelectParams& p, cudaStream_t st) {
  select_blocks_kernel<<<static_cast<unsigned>(static_cast<int64_t>(p.S) * p.Hkv), kSelectThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace pa
