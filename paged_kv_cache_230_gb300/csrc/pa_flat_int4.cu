// Instantiations of the flat decode (pa_flat.cuh) for 4-bit caches, and the
// joining of the pieces of contexts that several CTAs took.
#include <algorithm>

#include "pa_flat.cuh"

namespace pa {

cudaError_t launch_flat_int4(const FlatParams& p, int D, cudaStream_t st) { return launch_flat_kv<kInt4>(p, D, st); }

cudaError_t launch_flat_join(const FlatParams& p, int D, cudaStream_t st) {
  const int64_t contexts = static_cast<int64_t>(p.S) * p.heads;
  const int64_t joins = std::min<int64_t>(contexts, static_cast<int64_t>(p.nparts) * p.heads) * p.G * p.qlen;
  if (p.nparts == 1) return cudaSuccess;  // nothing is cut
  // few joins of many pieces each: 32 channels per CTA
  if (joins < p.sms) {
    return D == 64 ? launch_in_order(flat_join_kernel<64, 32>, static_cast<unsigned>(2 * joins), kJoinThreads, 0, st, p)
                   : launch_in_order(flat_join_kernel<128, 32>, static_cast<unsigned>(4 * joins), kJoinThreads, 0, st, p);
  }
  return D == 64 ? launch_in_order(flat_join_kernel<64, 64>, static_cast<unsigned>(joins), kJoinThreads, 0, st, p)
                 : launch_in_order(flat_join_kernel<128, 128>, static_cast<unsigned>(joins), kJoinThreads, 0, st, p);
}

}  // namespace pa
