// Instantiations of the flat decode (pa_flat.cuh) for e4m3 caches.
#include "pa_flat.cuh"

namespace pa {

cudaError_t launch_flat_e4m3(const FlatParams& p, int D, cudaStream_t st) { return launch_flat_kv<kE4M3>(p, D, st); }

}  // namespace pa
