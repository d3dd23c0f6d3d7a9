// Interface between the C entries of the cache-side operators (pa_ops_api.cu)
// and their kernels: norm + rotation + cache write, row-scaled caches, and the
// choice of blocks.  Not part of the ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

// Where the K and V rows of a call go.
struct RowSink {
  void* k_cache;
  void* v_cache;
  float* k_scales;  // row-scaled caches; nullptr otherwise
  float* v_scales;
  const int64_t* slot_mapping;
  int* err;
  int64_t num_slots;  // num_blocks * bs
  int Hkv, D, bs_log2;
  float kv_scale;
};

enum : int { kSink16 = 0, kSinkTensor = 1, kSinkRows = 2 };  // how rows are stored

struct NormRopeParams {
  void* q_out;
  const void* q;
  const void* key;
  const void* value;
  int64_t q_stride, key_stride, value_stride;  // elements
  const void* q_weight;  // nullptr: no norm
  const void* k_weight;
  const int64_t* positions;
  const float* cos_sin;
  int64_t num_positions;
  int T, Hq, rot, interleaved, bf16;
  int sms;    // of the device
  int tab16;  // set by the launcher: cos_sin is 16-byte aligned
  float eps;
  RowSink sink;
};
cudaError_t launch_norm_rope(const NormRopeParams& p, int sink_kind, cudaStream_t st);

struct CacheRowsParams {
  const void* key;
  const void* value;
  int T, bf16;
  int small;  // (token, head) pairs count in 32 bits (set by the launcher)
  RowSink sink;
};
cudaError_t launch_cache_rows(const CacheRowsParams& p, cudaStream_t st);

struct GatherRowsParams {
  void* k_dst;
  void* v_dst;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scales;
  const float* v_scales;
  const int64_t* ids;
  int* err;
  int64_t num_blocks;
  int n, rows, D, bf16;  // rows = Hkv * bs per block
};
cudaError_t launch_gather_rows(const GatherRowsParams& p, cudaStream_t st);

struct BoundsParams {
  void* bounds;
  const void* k_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  int* err;
  int64_t num_blocks;
  int S, maxB, Hkv, D, bs, num_new, kv_dtype;
  int touched;  // blocks that num_new tokens can lie in
};
cudaError_t launch_block_bounds(const BoundsParams& p, cudaStream_t st);

struct ScoresParams {
  float* scores;
  const void* q;
  const void* bounds;
  const int32_t* block_tables;
  const int32_t* context_lens;
  int* err;
  int64_t num_blocks;
  int S, maxB, Hq, Hkv, G, D, bs, q_bf16, kv_dtype;
  int sms;  // of the device
};
cudaError_t launch_block_scores(const ScoresParams& p, cudaStream_t st);

struct SelectParams {
  int32_t* tables;
  int32_t* lens;
  const float* scores;
  const int32_t* block_tables;
  const int32_t* context_lens;
  int* err;
  int S, maxB, Hkv, bs, n, sink, recent, sms;
};
cudaError_t launch_select_blocks(const SelectParams& p, cudaStream_t st);

}  // namespace pa
