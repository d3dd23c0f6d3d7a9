// Row-scaled E4M3 caches: writing a step's K and V rows with one scale per
// row, and reading whole blocks back as 16-bit values.  Both move each byte
// once and are bound by memory: every thread has its 16-byte loads in flight
// before it works on the first.  32768 tokens of 8 heads of 128 channels (407 MB
// in and out together): written in 31 us, 2048 blocks read back in 33.5, 0.94 of
// a plain copy's rate together; IEEE quotients for every code instead of a
// corrected reciprocal took 54 for the write.
#include "pa_launch.h"
#include "pa_pdl.cuh"
#include "pa_row_quant.cuh"
#include "pagedattn.h"

namespace pa {

namespace {

constexpr int kRowThreads = 256;

// A group of D / 16 lanes per (token, kv head) takes its K row and its V row: the
// two share their place.  A lane takes sixteen values of each, so that what a row
// costs whatever its lanes hold (its place, the reduction, the reciprocal) is
// shared by more of them: eight per lane took 35.7 us, at the issue rate's
// bound.  (Two (token, head) pairs per group: 30.4, but 2.4 us where 64 tokens
// take 1.8 with one.)
template <int D, bool BF16>
__global__ void __launch_bounds__(kRowThreads) cache_rows_kernel(const CacheRowsParams p) {
  constexpr int LPR = D / 16, GROUPS = kRowThreads / LPR;
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
    float x[2][8];
    widen8<BF16>(raw[v][0], x[0]);
    widen8<BF16>(raw[v][1], x[1]);
    bool plain;
    const float s = row_scale<LPR>(reinterpret_cast<const float(&)[16]>(x), plain);
    plain = plain && __all_sync(0xFFFFFFFFu, s >= kPlainScale || !live);
    if (!live) continue;
    uint2 q[2];
    if (plain) {
      const float y = __frcp_rn(s);
      q[0] = quantise8_as<true>(x[0], s, y);
      q[1] = quantise8_as<true>(x[1], s, y);
    } else {
      q[0] = quantise8_as<false>(x[0], s, 0.f);
      q[1] = quantise8_as<false>(x[1], s, 0.f);
    }
    uint8_t* codes = static_cast<uint8_t*>(v ? p.sink.v_cache : p.sink.k_cache) + row * D + 16 * c;
    *reinterpret_cast<uint4*>(codes) = make_uint4(q[0].x, q[0].y, q[1].x, q[1].y);
    if (c == 0) (v ? p.sink.v_scales : p.sink.k_scales)[row] = s;
  }
}

// CTA = (block i, K or V): eight codes -> 16 bytes per thread and piece, so a
// warp's stores are whole lines; kGatherAhead loads in flight per thread.
constexpr int kGatherAhead = 8;

template <int D, bool BF16>
__global__ void __launch_bounds__(kRowThreads) gather_rows_kernel(const GatherRowsParams p) {
  constexpr int PPR = D / 8;  // pieces per row
  pdl_enter();
  const int64_t i = blockIdx.x >> 1;
  const bool is_v = blockIdx.x & 1;
  const int64_t b = load_written(p.ids + i);
  if (b < 0 || b >= p.num_blocks) {
    if (!is_v && threadIdx.x == 0) atomicOr(p.err, PA_DEVERR_BLOCK_ID);
    return;
  }
  const float* scales = (is_v ? p.v_scales : p.k_scales) + b * p.rows;
  const uint2* src = reinterpret_cast<const uint2*>((is_v ? p.v_cache : p.k_cache) + b * p.rows * D);
  uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? p.v_dst : p.k_dst) + i * p.rows * D);
  const int pieces = p.rows * PPR;
  for (int q0 = threadIdx.x; q0 < pieces; q0 += kGatherAhead * kRowThreads) {
    uint2 u[kGatherAhead];
    float s[kGatherAhead];
#pragma unroll
    for (int n = 0; n < kGatherAhead; ++n) {
      const int q = q0 + n * kRowThreads;
      u[n] = q < pieces ? load_written(src + q) : make_uint2(0u, 0u);
      s[n] = q < pieces ? load_written(scales + q / PPR) : 0.f;
    }
#pragma unroll
    for (int n = 0; n < kGatherAhead; ++n) {
      const int q = q0 + n * kRowThreads;
      if (q >= pieces) break;
      float x[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w = j < 2 ? u[n].x : u[n].y;
        const __half2_raw h2 =
            __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * (j & 1))), __NV_E4M3);
        const float2 v = __half22float2(__half2(h2));
        x[2 * j] = v.x * s[n];
        x[2 * j + 1] = v.y * s[n];
      }
      dst[q] = narrow8<BF16>(x);
    }
  }
}

}  // namespace

cudaError_t launch_cache_rows(const CacheRowsParams& p0, cudaStream_t st) {
  CacheRowsParams p = p0;
  const int64_t pairs = static_cast<int64_t>(p.T) * p.sink.Hkv;
  const int groups = kRowThreads / (p.sink.D / 16);
  // 32-bit division of the pair's index, the last CTA's pairs past the end included
  p.small = pairs + groups <= UINT32_MAX;
  const unsigned grid = static_cast<unsigned>((pairs + groups - 1) / groups);
  auto kern = p.sink.D == 64 ? (p.bf16 ? cache_rows_kernel<64, true> : cache_rows_kernel<64, false>)
                             : (p.bf16 ? cache_rows_kernel<128, true> : cache_rows_kernel<128, false>);
  return launch_in_order(kern, grid, kRowThreads, 0, st, p);
}

cudaError_t launch_gather_rows(const GatherRowsParams& p, cudaStream_t st) {
  auto kern = p.D == 64 ? (p.bf16 ? gather_rows_kernel<64, true> : gather_rows_kernel<64, false>)
                        : (p.bf16 ? gather_rows_kernel<128, true> : gather_rows_kernel<128, false>);
  return launch_in_order(kern, 2u * static_cast<unsigned>(p.n), kRowThreads, 0, st, p);
}

}  // namespace pa
