// Row-scaled E4M3 caches: writing a step's K and V rows with one scale per
// row, and reading whole blocks back as 16-bit values.  Both move each byte
// once and are bound by memory: every thread has four independent 16-byte
// loads in flight before it works on the first.  32768 tokens of 8 heads of 128
// channels (406 MB in and out together): written in 35.7 us, 2048 blocks read
// back in 33.5, 0.88 of a plain copy's rate; IEEE quotients for every code
// instead of a corrected reciprocal took 54 for the write.
#include "pa_launch.h"
#include "pa_pdl.cuh"
#include "pa_row_quant.cuh"
#include "pagedattn.h"

namespace pa {

namespace {

constexpr int kRowThreads = 256;
constexpr int kAhead = 2;  // pairs of rows

// Groups of D / 8 lanes per (token, kv head), its K row and its V row: the two
// share their place.  A CTA takes kAhead pairs per group, consecutive groups
// on consecutive heads.
template <int D, bool BF16>
__global__ void __launch_bounds__(kRowThreads) cache_rows_kernel(const CacheRowsParams p) {
  constexpr int LPR = D / 8, GROUPS = kRowThreads / LPR;
  pdl_enter();
  const int c = threadIdx.x % LPR, g = threadIdx.x / LPR;
  int64_t pair = static_cast<int64_t>(blockIdx.x) * (kAhead * GROUPS) + g;  // t * Hkv + h
  const int64_t total = static_cast<int64_t>(p.T) * p.sink.Hkv;
  // (token, head) of the first pair by one division, of the others by steps of GROUPS pairs
  int64_t t = p.small ? static_cast<uint32_t>(pair) / static_cast<uint32_t>(p.sink.Hkv) : pair / p.sink.Hkv;
  int h = static_cast<int>(pair - t * p.sink.Hkv);
  const uint4* key = static_cast<const uint4*>(p.key) + pair * LPR + c;
  const uint4* value = static_cast<const uint4*>(p.value) + pair * LPR + c;
  uint4 raw[kAhead][2];
  int64_t slot[kAhead];
  int head[kAhead];
#pragma unroll
  for (int n = 0; n < kAhead; ++n) {
    slot[n] = -1;
    head[n] = h;
    raw[n][0] = raw[n][1] = make_uint4(0u, 0u, 0u, 0u);
    if (pair < total) {
      slot[n] = load_written(p.sink.slot_mapping + t);
      raw[n][0] = __ldlu(key + n * GROUPS * LPR);  // read once (32768 tokens: 38.6 us by plain loads, 35.7)
      raw[n][1] = __ldlu(value + n * GROUPS * LPR);
    }
    pair += GROUPS;
    t += p.step_tokens;
    h += p.step_heads;
    if (h >= p.sink.Hkv) {
      h -= p.sink.Hkv;
      ++t;
    }
  }
#pragma unroll
  for (int n = 0; n < kAhead; ++n) {
    const bool in_pool = slot[n] < p.sink.num_slots;
    if (!in_pool && head[n] == 0 && c == 0) atomicOr(p.sink.err, PA_DEVERR_SLOT);
    const bool live = slot[n] >= 0 && in_pool;
    const int64_t row = live ? row_index(p.sink, slot[n], head[n]) : 0;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      float x[8];
      widen8<BF16>(raw[n][v], x);
      store_row<D, kSinkRows, BF16, true>(p.sink, v == 1, row, 2 * c, 2 * c + 1, c == 0, x, live);
    }
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
  const int groups = kRowThreads / (p.sink.D / 8), per_cta = kAhead * groups;
  p.step_tokens = groups / p.sink.Hkv;
  p.step_heads = groups % p.sink.Hkv;
  // 32-bit division of the pair's index, the last CTA's pairs past the end included
  p.small = pairs + per_cta <= UINT32_MAX;
  const unsigned grid = static_cast<unsigned>((pairs + per_cta - 1) / per_cta);
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
