// Rows of head_dim values held eight per lane by D / 8 neighbouring lanes:
// widening, reductions over the row's lanes, and storing a K or V row in the
// three forms of a cache (16-bit, E4M3 per tensor, E4M3 row-scaled).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "pa_ops.h"

namespace pa {

constexpr float kE4M3Max = 448.f;
constexpr float kLeastScale = 1.17549435e-38f;  // 2^-126: scales stay normal, x / scale finite

template <bool BF16>
__device__ __forceinline__ void widen8(const uint4 u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = v.x;
      x[2 * i + 1] = v.y;
    }
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 narrow8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    } else {
      const __half2 v = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// e4m3_rne_satfinite(x / s), IEEE division.
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float s) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 v = make_float2(__fdiv_rn(x[4 * i + 2 * j], s), __fdiv_rn(x[4 * i + 2 * j + 1], s));
      w[i] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3)) << (16 * j);
    }
  }
  return make_uint2(w[0], w[1]);
}

// The row's scale from this lane's eight values and the row's other lanes:
// the largest finite magnitude / 448, at least 2^-126.
template <int LPR>
__device__ __forceinline__ float row_scale(const float (&x)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(x[i]);
    m = a <= 3.40282347e38f ? fmaxf(m, a) : m;  // false for infinities and NaN
  }
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  return fmaxf(__fdiv_rn(m, kE4M3Max), kLeastScale);
}

// Stores lane `c`'s piece of row (slot, head h).  All lanes of the warp call
// this; `live` lanes store.
template <int D, int KIND, bool BF16>
__device__ __forceinline__ void store_row(const RowSink& p, bool is_value, int64_t slot, int h, int c,
                                          const float (&x)[8], bool live) {
  constexpr int LPR = D / 8;
  float s = p.kv_scale;
  if constexpr (KIND == kSinkRows) s = row_scale<LPR>(x);
  if (!live) return;
  const int64_t row = ((slot / p.bs) * p.Hkv + h) * p.bs + slot % p.bs;
  void* cache = is_value ? p.v_cache : p.k_cache;
  if constexpr (KIND == kSink16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(cache) + row * D + c * 8) = narrow8<BF16>(x);
  } else {
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + row * D + c * 8) = quantise8(x, s);
    if constexpr (KIND == kSinkRows) {
      if (c == 0) (is_value ? p.v_scales : p.k_scales)[row] = s;
    }
  }
}

}  // namespace pa
