// Instantiations of the flat decode (pa_flat.cuh) for 4-bit caches, and the
// joining of the pieces of contexts that several CTAs took.
#include "pa_flat.cuh"

namespace pa {

cudaError_t launch_flat_int4(const FlatParams& p, int D, cudaStream_t st) { return launch_flat_kv<kInt4>(p, D, st); }

cudaError_t launch_flat_join(const FlatParams& p, int D, cudaStream_t st) {
  const int64_t contexts = static_cast<int64_t>(p.S) * p.heads;
  const unsigned joins = static_cast<unsigned>(contexts < p.ncta ? contexts : p.ncta);
  const unsigned grid = joins * static_cast<unsigned>(p.G * p.qlen);
  return D == 64 ? launch_in_order(flat_join_kernel<64>, grid, 128, 0, st, p)
                 : launch_in_order(flat_join_kernel<128>, grid, 128, 0, st, p);
}

}  // namespace pa
