// Decode with a block table per (sequence, cache head), E4M3 caches.
#include "pa_decode.cuh"

namespace pa {

cudaError_t launch_decode_heads_fp8(const DecodeParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV,
                              int head_dim, cudaStream_t st) {
  return launch_decode_kv<kE4M3, kHeadTables>(p, tmK, tmV, head_dim, st);
}

}  // namespace pa
