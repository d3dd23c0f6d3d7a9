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

// A row's eight values per lane are two pieces of four channels, `pa` and `pb`
// (in pieces from the row's start); neighbouring pieces move as one.
// (Plain loads: a call may write its queries in place.)
template <bool JOINED>
__device__ __forceinline__ uint4 load_pieces(const uint16_t* row, int pa, int pb) {
  if constexpr (JOINED) return *reinterpret_cast<const uint4*>(row + 4 * pa);
  const uint2 a = *reinterpret_cast<const uint2*>(row + 4 * pa);
  const uint2 b = *reinterpret_cast<const uint2*>(row + 4 * pb);
  return make_uint4(a.x, a.y, b.x, b.y);
}
template <bool JOINED>
__device__ __forceinline__ void store_pieces(uint16_t* row, int pa, int pb, const uint4 u) {
  if constexpr (JOINED) {
    *reinterpret_cast<uint4*>(row + 4 * pa) = u;
  } else {
    *reinterpret_cast<uint2*>(row + 4 * pa) = make_uint2(u.x, u.y);
    *reinterpret_cast<uint2*>(row + 4 * pb) = make_uint2(u.z, u.w);
  }
}

// Index of row (slot, head h) among a cache's rows [NB, Hkv, bs].
__device__ __forceinline__ int64_t row_index(const RowSink& p, int64_t slot, int h) {
  return (((slot >> p.bs_log2) * p.Hkv + h) << p.bs_log2) + (slot & ((1 << p.bs_log2) - 1));
}

// Stores this lane's two pieces of a K or V row.  All lanes of the warp call
// this; `live` lanes store.  `first` is set in one lane of the row.
template <int D, int KIND, bool BF16, bool JOINED>
__device__ __forceinline__ void store_row(const RowSink& p, bool is_value, int64_t row, int pa, int pb, bool first,
                                          const float (&x)[8], bool live) {
  float s = p.kv_scale;
  if constexpr (KIND == kSinkRows) s = row_scale<D / 8>(x);
  if (!live) return;
  void* cache = is_value ? p.v_cache : p.k_cache;
  if constexpr (KIND == kSink16) {
    store_pieces<JOINED>(static_cast<uint16_t*>(cache) + row * D, pa, pb, narrow8<BF16>(x));
  } else {
    const uint2 q = quantise8(x, s);
    uint8_t* dst = static_cast<uint8_t*>(cache) + row * D;
    if constexpr (JOINED) {
      *reinterpret_cast<uint2*>(dst + 4 * pa) = q;
    } else {
      *reinterpret_cast<uint32_t*>(dst + 4 * pa) = q.x;
      *reinterpret_cast<uint32_t*>(dst + 4 * pb) = q.y;
    }
    if constexpr (KIND == kSinkRows) {
      if (first) (is_value ? p.v_scales : p.k_scales)[row] = s;
    }
  }
}

}  // namespace pa
