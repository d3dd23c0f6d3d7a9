// Interface between the C entries of the attention over 4-bit caches and
// through windows (pa_flat_api.cu) and its kernels.  Not part of the ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_ops.h"

namespace pa {

constexpr int kFlatWarps = 4;  // of a CTA, each with a part of its own
constexpr int kFlatThreads = 32 * kFlatWarps;
constexpr int kFlatTile = 64;      // tokens of a tile, at most
constexpr int kFlatColumns = 16;   // query columns of a warp at most
constexpr int kFlatCtasPerSm = 4;  // of any variant, at most

enum : int { kInt4 = 3 };  // beside kF16, kBF16, kE4M3 (pa_internal.h)

constexpr int kGroupChannels = 64;  // that share a scale and a least value

struct FlatParams {
  void* out;                    // [S, qlen, Hq, D] of the q type
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const void* k_params;         // 4-bit caches: [NB, cache heads, bs, D / 64, 2]
  const void* v_params;
  const int32_t* block_tables;  // [S, maxB]
  const int32_t* context_lens;  // [S]
  // a context is what one (sequence, head) attends to
  float* ws_o;                  // [2 nparts heads][kFlatColumns][D] sums of contexts' pieces
  float* ws_ml;                 // [2 nparts heads][kFlatColumns][2]
  int4* ws_joins;               // of several parts, [min(nparts heads, contexts)]: context, pieces, first piece's slot
  int* err;
  uint32_t blocks32;  // of the pool, at most 2^31 - 1 (ids are int32)
  int S, Hq, heads;  // heads: cache heads x head_div
  int head_div;      // contexts that share a cache head's query heads
  int G;             // query heads of each
  int bs_log2, maxB, qlen, q_bf16;
  int window;  // 0: none
  int sinks;
  // set by the launcher
  int cluster;     // CTAs that share a context; 0: the contexts are laid on a line
  int nparts;      // of the line, each of one warp per head
  int least_part;  // places of a part, at least
  int gap;         // places between contexts
  int by_context;  // joins are indexed by context, else by part and head
  int sms;
  uint32_t flip;   // 0xFFFF0000
  int negative;    // the scale is: scale_log2 is its size
  float scale_log2, kv_scale;
};

// kv: kF16, kBF16 or kE4M3 (pa_internal.h), or kInt4
cudaError_t launch_flat_f16(const FlatParams& p, int D, cudaStream_t st);
cudaError_t launch_flat_bf16(const FlatParams& p, int D, cudaStream_t st);
cudaError_t launch_flat_e4m3(const FlatParams& p, int D, cudaStream_t st);
cudaError_t launch_flat_int4(const FlatParams& p, int D, cudaStream_t st);
// Joins the pieces of contexts that several warps took.
cudaError_t launch_flat_join(const FlatParams& p, int D, cudaStream_t st);

// Warps that leave pieces on a GPU of `sms` multiprocessors, at most.
inline size_t flat_most_warps(int sms) { return static_cast<size_t>(sms) * kFlatCtasPerSm * kFlatWarps; }
// Workspace: the joins, then the pieces' (m, l), then their sums.
inline size_t flat_workspace_bytes(int sms, int D) {
  const size_t n = flat_most_warps(sms);
  return n * sizeof(int4) + 2 * n * kFlatColumns * (2 + D) * sizeof(float);
}

struct CacheInt4Params {
  const void* key;
  const void* value;
  int T, bf16;
  int small;  // (token, head) pairs count in 32 bits (set by the launcher)
  RowSink sink;  // k_scales and v_scales: the parameters
};
cudaError_t launch_cache_int4(const CacheInt4Params& p, cudaStream_t st);

// GatherRowsParams with the parameters in place of the scales.
cudaError_t launch_gather_int4(const GatherRowsParams& p, cudaStream_t st);

}  // namespace pa
