// 4-bit caches: writing a step's K and V rows, and reading whole blocks back as
// 16-bit values.
//
// 64 neighbouring channels share a scale and a least value, both bfloat16:
//   low   = the group's smallest value, rounded down
//   scale = max((largest - low) / 15 rounded to nearest, 2^-126)
//   code  = (x - low) / scale rounded to nearest even, 0 .. 15
// With low rounded down every value lies at or above it, and the scale is off by 2^-8 of
// itself at most, so the largest value lies within a seventeenth of a scale of low + 15
// scale: every value is off by half a scale at most, however far the group lies from 0.
//
// Both move each byte once; memory bounds reading back (2048 blocks of 16 tokens, 8 heads
// of 128: 28.4 us for 25 of copying), instructions the write (below).
#include <math_constants.h>

#include "pa_cache_row.cuh"
#include "pa_flat.h"
#include "pa_launch.h"
#include "pa_pdl.cuh"
#include "pa_row_quant.cuh"
#include "pagedattn.h"

namespace pa {

namespace {

constexpr int kInt4Threads = 256;
constexpr float kMostBf16 = 3.38953139e38f;
constexpr float kMostF32 = 3.40282347e38f;

__device__ __forceinline__ float bf16_bits(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }

// The larger and the smaller of two pairs of 16-bit numbers, NaN where either is.
template <bool BF16>
__device__ __forceinline__ uint32_t larger2(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (BF16)
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <bool BF16>
__device__ __forceinline__ uint32_t smaller2(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (BF16)
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// A group of D / 16 lanes per (token, kv head) takes its K row and its V row, 16
// channels per lane: four lanes a group of channels.  The instructions bound it:
// extremes are taken from pairs as they are stored, and codes gathered by
// multiply-adds, the other pipe than comparisons and logic take (32768 tokens of 8
// heads of 128 bf16 channels: from widened values and by shifts 37.4 us, so 34.0).
template <int D, bool BF16>
__global__ void __launch_bounds__(kInt4Threads) cache_int4_kernel(const CacheInt4Params p) {
  constexpr int LPR = D / 16, GROUPS = kInt4Threads / LPR;
  pdl_enter();
  const int c = threadIdx.x % LPR;
  const int64_t pair = static_cast<int64_t>(blockIdx.x) * GROUPS + threadIdx.x / LPR;  // t * Hkv + h
  const int64_t total = static_cast<int64_t>(p.T) * p.sink.Hkv;
  const int64_t t = p.small ? static_cast<uint32_t>(pair) / static_cast<uint32_t>(p.sink.Hkv) : pair / p.sink.Hkv;
  const int h = static_cast<int>(pair - t * p.sink.Hkv);
  const uint4* in[2] = {static_cast<const uint4*>(p.key) + (pair * LPR + c) * 2,
                        static_cast<const uint4*>(p.value) + (pair * LPR + c) * 2};
  int64_t slot = -1;
  uint4 raw[2][2];
#pragma unroll
  for (int v = 0; v < 2; ++v) raw[v][0] = raw[v][1] = make_uint4(0u, 0u, 0u, 0u);
  if (pair < total) {
    slot = load_written(p.sink.slot_mapping + t);
#pragma unroll
    for (int v = 0; v < 2; ++v) {  // read once
      raw[v][0] = __ldlu(in[v]);
      raw[v][1] = __ldlu(in[v] + 1);
    }
  }
  const bool in_pool = slot < p.sink.num_slots;
  if (!in_pool && h == 0 && c == 0) atomicOr(p.sink.err, PA_DEVERR_SLOT);
  const bool live = slot >= 0 && in_pool;
  const int64_t row = live ? row_index(p.sink, slot, h) : 0;
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    const uint32_t pairs[8] = {raw[v][0].x, raw[v][0].y, raw[v][0].z, raw[v][0].w,
                               raw[v][1].x, raw[v][1].y, raw[v][1].z, raw[v][1].w};
    float x[16];
    widen8<BF16>(raw[v][0], reinterpret_cast<float(&)[8]>(x[0]));
    widen8<BF16>(raw[v][1], reinterpret_cast<float(&)[8]>(x[8]));
    uint32_t top = pairs[0], bottom = pairs[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      top = larger2<BF16>(top, pairs[i]);
      bottom = smaller2<BF16>(bottom, pairs[i]);
    }
    // (largest, -least) of the lane, then of the group's four lanes
    top = larger2<BF16>(top, __byte_perm(top, top, 0x1032));
    bottom = smaller2<BF16>(bottom, __byte_perm(bottom, bottom, 0x1032));
    uint32_t both = __byte_perm(top, bottom, 0x5410) ^ 0x80000000u;
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) both = larger2<BF16>(both, __shfl_xor_sync(0xFFFFFFFFu, both, o));
    float most = widen16(both & 0xFFFFu, BF16 ? kBF16 : kF16), least = -widen16(both >> 16, BF16 ? kBF16 : kF16);
    // moderate finite values and scales: the quotient by div_by, between 0 and 15.1
    bool plain = __all_sync(0xFFFFFFFFu, fabsf(most) <= kPlainRange && fabsf(least) <= kPlainRange);
    int nan = 0;
    if (!plain) {
      least = CUDART_INF_F;
      most = -CUDART_INF_F;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        nan |= x[i] != x[i] ? 1 : 0;
        if (fabsf(x[i]) <= kMostF32) {
          least = fminf(least, x[i]);
          most = fmaxf(most, x[i]);
        }
      }
#pragma unroll
      for (int o = 1; o <= 2; o <<= 1) {
        nan |= __shfl_xor_sync(0xFFFFFFFFu, nan, o);
        least = fminf(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
      }
    }
    if (least > most) least = most = 0.f;  // nothing finite
    const uint16_t low16 = __bfloat16_as_ushort(__float2bfloat16_rd(fmaxf(least, -kMostBf16)));
    const float low = bf16_bits(low16);
    const float fifteenth = __fdiv_rn(fminf(most - low, kMostF32), 15.f);
    uint16_t scale16 = __bfloat16_as_ushort(__float2bfloat16_rn(fmaxf(fifteenth, kLeastScale)));
    const float scale = bf16_bits(scale16);
    plain = plain && __all_sync(0xFFFFFFFFu, scale >= kPlainScale || !live);
    uint32_t w[2] = {0u, 0u};
    constexpr float kWhole = 12582912.f;  // 1.5 * 2^23: its sum with 0 .. 15 is rounded to whole numbers
    constexpr uint32_t kWholeBits = 0x4B400000u;
    if (plain) {
      // the sums' bits are kWhole's plus the code: times the nibble's place and added up,
      // with what kWhole's bits make of it taken off beforehand
      constexpr uint32_t kPlaces = 0x11111111u;
      const float y = __frcp_rn(scale);
      w[0] = w[1] = 0u - kWholeBits * kPlaces;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        w[i / 8] += __float_as_uint(div_by(x[i] - low, scale, y) + kWhole) * (1u << (4 * (i % 8 / 2) + 16 * (i & 1)));
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float q = fminf(fmaxf(__fdiv_rn(x[i] - low, scale), 0.f), 15.f);  // a NaN as 0
        const uint32_t code = __float_as_uint(q + kWhole) & 15u;
        w[i / 8] |= code << (4 * (i % 8 / 2) + 16 * (i & 1));
      }
      if (nan) scale16 = 0x7FFFu;  // the group reads as NaN
    }
    if (!live) continue;
    uint8_t* codes = static_cast<uint8_t*>(v ? p.sink.v_cache : p.sink.k_cache) + row * (D / 2) + 8 * c;
    *reinterpret_cast<uint2*>(codes) = make_uint2(w[0], w[1]);
    uint32_t* params = reinterpret_cast<uint32_t*>(v ? p.sink.v_scales : p.sink.k_scales) + row * (D / kGroupChannels);
    if (c % 4 == 0) params[c / 4] = scale16 | static_cast<uint32_t>(low16) << 16;
  }
}

// Two 16-bit numbers, infinities as the largest finite one.
template <bool BF16>
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  constexpr uint32_t kMost = BF16 ? 0x7F7F7F7Fu : 0x7BFF7BFFu;
  return larger2<BF16>(smaller2<BF16>(w, kMost), kMost | 0x80008000u);
}

// CTA = (block i, K or V): eight codes -> 16 bytes per thread and piece, so a
// warp's stores are whole lines; kGatherAhead loads in flight per thread.
constexpr int kGatherAhead = 8;

template <int D, bool BF16>
__global__ void __launch_bounds__(kInt4Threads) gather_int4_kernel(const GatherRowsParams p) {
  constexpr int PPR = D / 8, PPG = kGroupChannels / 8;  // pieces per row, per group of channels
  pdl_enter();
  const int64_t i = blockIdx.x >> 1;
  const bool is_v = blockIdx.x & 1;
  const int64_t b = load_written(p.ids + i);
  if (b < 0 || b >= p.num_blocks) {
    if (!is_v && threadIdx.x == 0) atomicOr(p.err, PA_DEVERR_BLOCK_ID);
    return;
  }
  const uint32_t* params = reinterpret_cast<const uint32_t*>(is_v ? p.v_scales : p.k_scales) + b * p.rows * (PPR / PPG);
  const uint32_t* src = reinterpret_cast<const uint32_t*>(is_v ? p.v_cache : p.k_cache) + b * p.rows * PPR;
  uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? p.v_dst : p.k_dst) + i * p.rows * D);
  const int pieces = p.rows * PPR;
  for (int q0 = threadIdx.x; q0 < pieces; q0 += kGatherAhead * kInt4Threads) {
    uint32_t u[kGatherAhead], s[kGatherAhead];
#pragma unroll
    for (int n = 0; n < kGatherAhead; ++n) {
      const int q = q0 + n * kInt4Threads;
      u[n] = q < pieces ? load_written(src + q) : 0u;
      s[n] = q < pieces ? load_written(params + q / PPG) : 0u;
    }
#pragma unroll
    for (int n = 0; n < kGatherAhead; ++n) {
      const int q = q0 + n * kInt4Threads;
      if (q >= pieces) break;
      const float scale = __uint_as_float(s[n] << 16), low = __uint_as_float(s[n] & 0xFFFF0000u);
      float x[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // a nibble in the last bits of 2^23 and that subtracted
        x[2 * k] = fmaf(__uint_as_float((u[n] >> (4 * k) & 15u) | 0x4B000000u) - 8388608.f, scale, low);
        x[2 * k + 1] = fmaf(__uint_as_float((u[n] >> (4 * k + 16) & 15u) | 0x4B000000u) - 8388608.f, scale, low);
      }
      uint4 y = narrow8<BF16>(x);
      // a least value rounded down, or fifteen scales rounded up, may lie past the largest
      // number of 16 bits where the value that was written did not
      constexpr float kMost = BF16 ? kMostBf16 : 65504.f;
      if (!(fabsf(low) <= kMost && fabsf(fmaf(15.f, scale, low)) <= kMost))
        y = make_uint4(finite2<BF16>(y.x), finite2<BF16>(y.y), finite2<BF16>(y.z), finite2<BF16>(y.w));
      dst[q] = y;
    }
  }
}

}  // namespace

cudaError_t launch_cache_int4(const CacheInt4Params& p0, cudaStream_t st) {
  CacheInt4Params p = p0;
  const int64_t pairs = static_cast<int64_t>(p.T) * p.sink.Hkv;
  const int groups = kInt4Threads / (p.sink.D / 16);
  // 32-bit division of the pair's index, the last CTA's pairs past the end included
  p.small = pairs + groups <= UINT32_MAX;
  const unsigned grid = static_cast<unsigned>((pairs + groups - 1) / groups);
  auto kern = p.sink.D == 64 ? (p.bf16 ? cache_int4_kernel<64, true> : cache_int4_kernel<64, false>)
                             : (p.bf16 ? cache_int4_kernel<128, true> : cache_int4_kernel<128, false>);
  return launch_in_order(kern, grid, kInt4Threads, 0, st, p);
}

cudaError_t launch_gather_int4(const GatherRowsParams& p, cudaStream_t st) {
  auto kern = p.D == 64 ? (p.bf16 ? gather_int4_kernel<64, true> : gather_int4_kernel<64, false>)
                        : (p.bf16 ? gather_int4_kernel<128, true> : gather_int4_kernel<128, false>);
  return launch_in_order(kern, 2u * static_cast<unsigned>(p.n), kInt4Threads, 0, st, p);
}

}  // namespace pa
