// Wide loads from the shared memory of a cluster's CTAs (addresses by peer_shared,
// or of the CTA's own).
#pragma once

#include <stdint.h>

namespace pa {

__device__ __forceinline__ float2 load_peer2(uint32_t addr) {
  float2 y;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(y.x), "=f"(y.y) : "r"(addr) : "memory");
  return y;
}
__device__ __forceinline__ float4 load_peer4(uint32_t addr) {
  float4 y;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(y.x), "=f"(y.y), "=f"(y.z), "=f"(y.w)
               : "r"(addr)
               : "memory");
  return y;
}

}  // namespace pa
