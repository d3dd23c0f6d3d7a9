// Instantiations of the flat decode (pa_flat.cuh) for bf16 caches.
#include "pa_flat.cuh"

namespace pa {

cudaError_t launch_flat_bf16(const FlatParams& p, int D, cudaStream_t st) { return launch_flat_kv<kBF16>(p, D, st); }

}  // namespace pa
