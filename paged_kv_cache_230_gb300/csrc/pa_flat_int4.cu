// Instantiations of the flat decode (pa_flat.cuh) for 4-bit caches, and the
// joining of the pieces of contexts that several CTAs took.
#include <algorithm>

#include "pa_flat.cuh"

namespace pa {

cudaError_t launch_flat_int4(const FlatParams& p, int D, cudaStream_t st) {
  return p.q_bf16 ? launch_flat_kv<kInt4, false>(p, D, st) : launch_flat_kv<kInt4, true>(p, D, st);
}

cudaError_t launch_flat_join(const FlatParams& p, int D, cudaStream_t st) {
  const int64_t contexts = static_cast<int64_t>(p.S) * p.heads;
  const int64_t joins = std::min<int64_t>(contexts, static_cast<int64_t>(p.nparts) * p.heads);
  if (p.nparts == 1) return cudaSuccess;  // nothing is cut
  if (p.nparts / 6 >= p.S) {  // contexts of many pieces
    const unsigned grid = static_cast<unsigned>(joins * p.G * p.qlen);
    return D == 64 ? launch_in_order(flat_join_kernel<64, true>, grid, kJoinThreads, 0, st, p)
                   : launch_in_order(flat_join_kernel<128, true>, grid, kJoinThreads, 0, st, p);
  }
  return D == 64 ? launch_in_order(flat_join_kernel<64, false>, static_cast<unsigned>(joins), kJoinThreads, 0, st, p)
                 : launch_in_order(flat_join_kernel<128, false>, static_cast<unsigned>(joins), kJoinThreads, 0, st, p);
}

}  // namespace pa
