// Decode with a block table per (sequence, cache head), bf16 caches.
#include "pa_decode.cuh"

namespace pa {

cudaError_t launch_decode_heads_bf16(const DecodeParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV,
                              int head_dim, cudaStream_t st) {
  return launch_decode_kv<kBF16, kHeadTables>(p, tmK, tmV, head_dim, st);
}

}  // namespace pa
