// Decode with a block table per (sequence, cache head), f16 caches.
#include "pa_decode.cuh"

namespace pa {

cudaError_t launch_decode_heads_f16(const DecodeParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV,
                              int head_dim, cudaStream_t st) {
  return launch_decode_kv<kF16, kHeadTables>(p, tmK, tmV, head_dim, st);
}

}  // namespace pa
