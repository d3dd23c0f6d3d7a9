// Row-scaled E4M3 caches: writing a step's K and V rows with one scale per
// row, and reading whole blocks back as 16-bit values.  Both move each byte
// once and are bound by memory.
#include "pa_row_quant.cuh"
#include "pagedattn.h"

namespace pa {

namespace {

constexpr int kRowThreads = 256;

// A group of D / 8 lanes per (token, kv head, K or V) row.
template <int D, bool BF16>
__global__ void __launch_bounds__(kRowThreads) cache_rows_kernel(const CacheRowsParams p) {
  constexpr int LPR = D / 8;
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
  const int c = static_cast<int>(idx % LPR);
  const int64_t row = idx / LPR;  // (t * 2 + K or V) * Hkv + h
  const int h = static_cast<int>(row % p.sink.Hkv);
  const int64_t tv = row / p.sink.Hkv;
  const bool is_v = tv & 1, on = (tv >> 1) < p.T;
  const int64_t t = tv >> 1;
  const int64_t slot = on ? p.sink.slot_mapping[t] : -1;
  if (slot >= p.sink.num_slots && !is_v && h == 0 && c == 0) atomicOr(p.sink.err, PA_DEVERR_SLOT);
  const bool live = slot >= 0 && slot < p.sink.num_slots;
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = 0.f;
  if (live)
    widen8<BF16>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(is_v ? p.value : p.key) +
                                                 (t * p.sink.Hkv + h) * D + c * 8),
                 x);
  store_row<D, kSinkRows, BF16>(p.sink, is_v, slot, h, c, x, live);
}

// 16 codes and their row's scale -> 32 bytes, per thread.
template <int D, bool BF16>
__global__ void __launch_bounds__(kRowThreads) gather_rows_kernel(const GatherRowsParams p) {
  constexpr int PPR = D / 16;  // pieces per row
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
  const int64_t row = idx / PPR;  // (i * 2 + K or V) * rows + row in the block
  const int piece = static_cast<int>(idx % PPR);
  const int64_t iv = row / p.rows;
  const int r = static_cast<int>(row % p.rows);
  const bool is_v = iv & 1;
  const int64_t i = iv >> 1;
  if (i >= p.n) return;
  const int64_t b = p.ids[i];
  if (b < 0 || b >= p.num_blocks) {
    if (!is_v && r == 0 && piece == 0) atomicOr(p.err, PA_DEVERR_BLOCK_ID);
    return;
  }
  const int64_t src = b * p.rows + r;
  const float s = __ldg((is_v ? p.v_scales : p.k_scales) + src);
  const uint4 u = __ldg(reinterpret_cast<const uint4*>((is_v ? p.v_cache : p.k_cache) + src * D) + piece);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? p.v_dst : p.k_dst) + (i * p.rows + r) * D) +
               2 * piece;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2_raw h2 = __nv_cvt_fp8x2_to_halfraw2(
          static_cast<__nv_fp8x2_storage_t>(w[2 * k + j / 2] >> (16 * (j & 1))), __NV_E4M3);
      const float2 v = __half22float2(__half2(h2));
      x[2 * j] = v.x * s;
      x[2 * j + 1] = v.y * s;
    }
    dst[k] = narrow8<BF16>(x);
  }
}

}  // namespace

cudaError_t launch_cache_rows(const CacheRowsParams& p, cudaStream_t st) {
  const int64_t total = static_cast<int64_t>(p.T) * p.sink.Hkv * 2 * (p.sink.D / 8);
  const unsigned grid = static_cast<unsigned>((total + kRowThreads - 1) / kRowThreads);
  if (p.sink.D == 64)
    p.bf16 ? cache_rows_kernel<64, true><<<grid, kRowThreads, 0, st>>>(p)
           : cache_rows_kernel<64, false><<<grid, kRowThreads, 0, st>>>(p);
  else
    p.bf16 ? cache_rows_kernel<128, true><<<grid, kRowThreads, 0, st>>>(p)
           : cache_rows_kernel<128, false><<<grid, kRowThreads, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_gather_rows(const GatherRowsParams& p, cudaStream_t st) {
  const int64_t total = static_cast<int64_t>(p.n) * 2 * p.rows * (p.D / 16);
  const unsigned grid = static_cast<unsigned>((total + kRowThreads - 1) / kRowThreads);
  if (p.D == 64)
    p.bf16 ? gather_rows_kernel<64, true><<<grid, kRowThreads, 0, st>>>(p)
           : gather_rows_kernel<64, false><<<grid, kRowThreads, 0, st>>>(p);
  else
    p.bf16 ? gather_rows_kernel<128, true><<<grid, kRowThreads, 0, st>>>(p)
           : gather_rows_kernel<128, false><<<grid, kRowThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace pa
