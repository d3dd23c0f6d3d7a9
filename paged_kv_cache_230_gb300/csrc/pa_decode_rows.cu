// Decode over E4M3 caches with one scale per (token, head) row.
#include "pa_decode.cuh"

namespace pa {

cudaError_t launch_decode_rows(const DecodeParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV, int head_dim,
                               cudaStream_t st) {
  return launch_decode_kv<kE4M3, kRowScaled>(p, tmK, tmV, head_dim, st);
}

}  // namespace pa
