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

// x / s rounded to nearest as IEEE division does, from y = 1 / s rounded to
// nearest: q = x y is within a unit in the last place, its remainder x - q s is
// exact in one fused multiply-add, and adding remainder * y rounds correctly
// (Markstein's theorem).  For finite x and where nothing overflows or loses
// bits below 2^-149: s at least 2^-90 keeps every bit of the remainder of any
// x that reaches an E4M3 code (|x / s| >= 2^-10).
__device__ __forceinline__ float div_by(float x, float s, float y) {
  const float q = x * y;
  return fmaf(fmaf(-q, s, x), y, q);
}

// e4m3_rne_satfinite(x / s).  PLAIN: div_by applies.
template <bool PLAIN>
__device__ __forceinline__ uint2 quantise8_as(const float (&x)[8], float s, float y) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float a = x[4 * i + 2 * j], b = x[4 * i + 2 * j + 1];
      const float2 v = PLAIN ? make_float2(div_by(a, s, y), div_by(b, s, y))
                             : make_float2(__fdiv_rn(a, s), __fdiv_rn(b, s));
      w[i] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3)) << (16 * j);
    }
  }
  return make_uint2(w[0], w[1]);
}

constexpr float kPlainScale = 8.07793567e-28f;  // 2^-90
constexpr float kPlainRange = 1.15292150e18f;   // 2^60

__device__ __forceinline__ float magnitude_max(float m, float x) {  // max(m, |x|), NaN if either is
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(m), "f"(fabsf(x)));
  return y;
}

// The row's scale from this lane's N values and the row's other lanes:
// the largest finite magnitude / 448, at least 2^-126.  `finite`: whether all
// values of the warp's rows are.  All lanes of the warp call this.
template <int LPR, int N>
__device__ __forceinline__ float row_scale(const float (&x)[N], bool& finite) {
  constexpr float kMax = 3.40282347e38f;
  float m = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < N; ++i) m = magnitude_max(m, x[i]);
  finite = __all_sync(0xFFFFFFFFu, m <= kMax);
  if (!finite) {
    m = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float a = fabsf(x[i]);
      m = a <= kMax ? fmaxf(m, a) : m;
    }
  }
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  // quotients of 2^-126 and more are exact here (div_by), smaller ones not used
  return fmaxf(div_by(m, kE4M3Max, 1.f / kE4M3Max), kLeastScale);
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
  bool plain = false;
  if constexpr (KIND == kSinkRows) {
    s = row_scale<D / 8>(x, plain);
    plain = plain && __all_sync(0xFFFFFFFFu, s >= kPlainScale || !live);
  }
  if constexpr (KIND == kSinkTensor) {
    // a quotient that overflows has to saturate: moderate values and scales only
    float m = fabsf(x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = magnitude_max(m, x[i]);
    plain = s >= 1.f / kPlainRange && s <= kPlainRange && __all_sync(0xFFFFFFFFu, m <= kPlainRange || !live);
  }
  if (!live) return;
  void* cache = is_value ? p.v_cache : p.k_cache;
  if constexpr (KIND == kSink16) {
    store_pieces<JOINED>(static_cast<uint16_t*>(cache) + row * D, pa, pb, narrow8<BF16>(x));
  } else {
    const uint2 q = plain ? quantise8_as<true>(x, s, __frcp_rn(s)) : quantise8_as<false>(x, s, 0.f);
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
