// C entries of the 4-bit caches and of the decode through windows.
#include <algorithm>
#include <cmath>

#include "pa_flat.h"
#include "pa_host.h"

namespace {

using pa::host::aligned16;
using pa::host::error_word;
using pa::host::finish;

bool is16(int dtype) { return dtype == PA_F16 || dtype == PA_BF16; }

int check_int4(const pa_cache_desc* c, const void* k, const void* v, const void* kp, const void* vp) {
  const int rc = pa::host::check_cache_int4(c, k, v);
  if (rc) return rc;
  return kp && vp && aligned16(kp) && aligned16(vp) ? PA_OK : PA_ERR_INVALID_ARG;
}

struct FlatArgs {
  void* out;
  const void* q;
  int32_t q_dtype, num_seqs, num_q_tokens, num_q_heads;
  const void* k_cache;
  const void* v_cache;
  const void* k_params;
  const void* v_params;
  const pa_cache_desc* cache;
  const int32_t* block_tables;
  int32_t max_blocks;
  const int32_t* context_lens;
  float scale, kv_scale;
  int32_t window, sinks;
  void* workspace;
  size_t workspace_bytes;
};

// The cache itself has been checked.
int decode_flat(const FlatArgs& a, pa_stream_t stream) {
  const pa_cache_desc* c = a.cache;
  if (a.num_seqs < 0 || a.max_blocks <= 0 || a.num_q_heads <= 0 || a.num_q_tokens < 1 ||
      a.num_q_heads % c->num_kv_heads)
    return PA_ERR_INVALID_ARG;
  const int64_t capacity = static_cast<int64_t>(a.max_blocks) * c->block_size;
  if (capacity > INT32_MAX - pa::kFlatTile) return PA_ERR_INVALID_ARG;
  if (!is16(a.q_dtype) || a.num_q_heads / c->num_kv_heads > 128 || a.num_q_tokens > pa::kMaxGroup)
    return PA_ERR_UNSUPPORTED;
  if (!std::isfinite(a.scale) || a.sinks < 0) return PA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(a.num_seqs) * a.num_q_tokens * a.num_q_heads > INT32_MAX) return PA_ERR_INVALID_ARG;
  if (a.num_seqs == 0) return PA_OK;
  if (!a.out || !a.q || !a.block_tables || !a.context_lens || !aligned16(a.out) || !aligned16(a.q))
    return PA_ERR_INVALID_ARG;
  const int sms = pa::host::sms(), D = c->head_dim;
  if (!a.workspace || !aligned16(a.workspace) || a.workspace_bytes < pa::flat_workspace_bytes(sms, D))
    return PA_ERR_WORKSPACE;
  int* err = error_word();
  if (!err) return PA_ERR_CUDA;
  pa::FlatParams p{};
  p.out = a.out;
  p.q = a.q;
  p.k_cache = a.k_cache;
  p.v_cache = a.v_cache;
  p.k_params = a.k_params;
  p.v_params = a.v_params;
  p.block_tables = a.block_tables;
  p.context_lens = a.context_lens;
  const size_t warps = pa::flat_most_warps(sms);
  p.ws_joins = static_cast<int4*>(a.workspace);
  p.ws_ml = reinterpret_cast<float*>(p.ws_joins + warps);
  p.ws_o = p.ws_ml + 2 * warps * pa::kFlatColumns * 2;
  p.err = err;
  p.blocks32 = static_cast<uint32_t>(std::min<int64_t>(c->num_blocks, INT32_MAX));
  p.S = a.num_seqs;
  p.Hq = a.num_q_heads;
  const int G = a.num_q_heads / c->num_kv_heads;
  p.G = pa::host::heads_per_cta(G, a.num_q_tokens);
  p.head_div = G / p.G;
  p.heads = c->num_kv_heads * p.head_div;
  p.bs_log2 = c->block_size == 8 ? 3 : (c->block_size == 16 ? 4 : 5);
  p.maxB = a.max_blocks;
  p.qlen = a.num_q_tokens;
  p.q_bf16 = a.q_dtype == PA_BF16;
  // the window of a table that holds no more tokens than it is all of them
  p.window = a.window < capacity ? a.window : 0;
  p.sinks = p.window > 0 ? static_cast<int>(std::min<int64_t>(a.sinks, capacity)) : 0;
  p.sms = sms;
  p.flip = 0xFFFF0000u;
  p.negative = a.scale < 0.f;
  p.scale_log2 = static_cast<float>(std::fabs(static_cast<double>(a.scale)) * 1.4426950408889634);
  p.kv_scale = a.kv_scale;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (c->kv_dtype) {
    case PA_F16: e = pa::launch_flat_f16(p, D, st); break;
    case PA_BF16: e = pa::launch_flat_bf16(p, D, st); break;
    case PA_FP8_E4M3: e = pa::launch_flat_e4m3(p, D, st); break;
    default: e = pa::launch_flat_int4(p, D, st); break;
  }
  return finish(e, st);
}

}  // namespace

extern "C" {

int pa_reshape_and_cache_int4(const void* key, const void* value, int32_t in_dtype, int32_t num_tokens, void* k_cache,
                              void* v_cache, void* k_params, void* v_params, const pa_cache_desc* cache,
                              const int64_t* slot_mapping, pa_stream_t stream) {
  const int rc = check_int4(cache, k_cache, v_cache, k_params, v_params);
  if (rc) return rc;
  if (!is16(in_dtype)) return PA_ERR_UNSUPPORTED;
  if (num_tokens < 0) return PA_ERR_INVALID_ARG;
  if (num_tokens == 0) return PA_OK;
  if (!key || !value || !slot_mapping || !aligned16(key) || !aligned16(value)) return PA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(num_tokens) * cache->num_kv_heads > INT32_MAX * int64_t(16)) return PA_ERR_INVALID_ARG;
  int* err = error_word();
  if (!err) return PA_ERR_CUDA;
  pa::CacheInt4Params p{};
  p.key = key;
  p.value = value;
  p.T = num_tokens;
  p.bf16 = in_dtype == PA_BF16;
  p.sink.k_cache = k_cache;
  p.sink.v_cache = v_cache;
  p.sink.k_scales = static_cast<float*>(k_params);
  p.sink.v_scales = static_cast<float*>(v_params);
  p.sink.slot_mapping = slot_mapping;
  p.sink.err = err;
  p.sink.num_slots = cache->num_blocks * cache->block_size;
  p.sink.Hkv = cache->num_kv_heads;
  p.sink.D = cache->head_dim;
  p.sink.bs_log2 = cache->block_size == 8 ? 3 : (cache->block_size == 16 ? 4 : 5);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return finish(pa::launch_cache_int4(p, st), st);
}

int pa_gather_blocks_int4(void* k_dst, void* v_dst, int32_t dst_dtype, const void* k_cache, const void* v_cache,
                          const void* k_params, const void* v_params, const pa_cache_desc* cache,
                          const int64_t* block_ids, int32_t num, pa_stream_t stream) {
  const int rc = check_int4(cache, k_cache, v_cache, k_params, v_params);
  if (rc) return rc;
  if (!is16(dst_dtype)) return PA_ERR_UNSUPPORTED;
  if (num < 0) return PA_ERR_INVALID_ARG;
  if (num == 0) return PA_OK;
  if (!k_dst || !v_dst || !block_ids || !aligned16(k_dst) || !aligned16(v_dst)) return PA_ERR_INVALID_ARG;
  if (num > INT32_MAX / 2) return PA_ERR_INVALID_ARG;
  void* ids = nullptr;
  void* kd = nullptr;
  void* vd = nullptr;
  if (!pa::host::device_view(block_ids, &ids) || !pa::host::device_view(k_dst, &kd) ||
      !pa::host::device_view(v_dst, &vd))
    return PA_ERR_INVALID_ARG;
  int* err = error_word();
  if (!err) return PA_ERR_CUDA;
  pa::GatherRowsParams p{};
  p.k_dst = kd;
  p.v_dst = vd;
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.k_scales = static_cast<const float*>(k_params);
  p.v_scales = static_cast<const float*>(v_params);
  p.ids = static_cast<const int64_t*>(ids);
  p.err = err;
  p.num_blocks = cache->num_blocks;
  p.n = num;
  p.rows = cache->num_kv_heads * cache->block_size;
  p.D = cache->head_dim;
  p.bf16 = dst_dtype == PA_BF16;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return finish(pa::launch_gather_int4(p, st), st);
}

size_t pa_decode_flat_workspace_size(int32_t head_dim) {
  return head_dim == 64 || head_dim == 128 ? pa::flat_workspace_bytes(pa::host::sms(), head_dim) : 0;
}

int pa_decode_int4(void* out, const void* q, int32_t q_dtype, int32_t num_seqs, int32_t num_q_tokens,
                   int32_t num_q_heads, const void* k_cache, const void* v_cache, const void* k_params,
                   const void* v_params, const pa_cache_desc* cache, const int32_t* block_tables,
                   int32_t max_blocks_per_seq, const int32_t* context_lens, float scale, int32_t window,
                   int32_t num_sinks, void* workspace, size_t workspace_bytes, pa_stream_t stream) {
  const int rc = check_int4(cache, k_cache, v_cache, k_params, v_params);
  if (rc) return rc;
  if (window < 0) return PA_ERR_INVALID_ARG;
  return decode_flat({out, q, q_dtype, num_seqs, num_q_tokens, num_q_heads, k_cache, v_cache, k_params, v_params, cache,
                      block_tables, max_blocks_per_seq, context_lens, scale, 1.f, window, num_sinks, workspace,
                      workspace_bytes},
                     stream);
}

int pa_decode_window(void* out, const void* q, int32_t q_dtype, int32_t num_seqs, int32_t num_q_tokens,
                     int32_t num_q_heads, const void* k_cache, const void* v_cache, const pa_cache_desc* cache,
                     const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens, float scale,
                     float kv_scale, int32_t window, int32_t num_sinks, void* workspace, size_t workspace_bytes,
                     pa_stream_t stream) {
  int rc = pa::host::check_cache(cache, k_cache, v_cache);
  if (rc || (rc = pa::host::check_kv_scale(cache->kv_dtype, kv_scale))) return rc;
  if (cache->kv_dtype != PA_FP8_E4M3 && cache->kv_dtype != q_dtype) return PA_ERR_UNSUPPORTED;
  if (window < 1) return PA_ERR_INVALID_ARG;
  return decode_flat({out, q, q_dtype, num_seqs, num_q_tokens, num_q_heads, k_cache, v_cache, nullptr, nullptr, cache,
                      block_tables, max_blocks_per_seq, context_lens, scale, kv_scale, window, num_sinks, workspace,
                      workspace_bytes},
                     stream);
}

}  // extern "C"
