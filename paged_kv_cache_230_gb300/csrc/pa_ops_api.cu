// C entries of the cache-side operators: row-scaled caches, norm + rotation +
// cache write, and the choice of blocks with the decode over it.
#include <algorithm>
#include <cmath>

#include "pa_host.h"
#include "pa_ops.h"

namespace {

using pa::host::aligned16;
using pa::host::error_word;
using pa::host::finish;

bool is16(int dtype) { return dtype == PA_F16 || dtype == PA_BF16; }

int check_row_scales(const pa_cache_desc* c, const float* ks, const float* vs) {
  if (c->kv_dtype != PA_FP8_E4M3) return PA_ERR_UNSUPPORTED;
  return ks && vs && aligned16(ks) && aligned16(vs) ? PA_OK : PA_ERR_INVALID_ARG;
}

// Whether two byte ranges share a byte.
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + static_cast<uint64_t>(nb) && y < x + static_cast<uint64_t>(na);
}

pa::RowSink make_sink(void* k_cache, void* v_cache, float* k_scales, float* v_scales, const pa_cache_desc* cache,
                      const int64_t* slot_mapping, float kv_scale, int* err) {
  pa::RowSink s{};
  s.k_cache = k_cache;
  s.v_cache = v_cache;
  s.k_scales = k_scales;
  s.v_scales = v_scales;
  s.slot_mapping = slot_mapping;
  s.err = err;
  s.num_slots = cache->num_blocks * cache->block_size;
  s.Hkv = cache->num_kv_heads;
  s.D = cache->head_dim;
  s.bs_log2 = cache->block_size == 8 ? 3 : (cache->block_size == 16 ? 4 : 5);
  s.kv_scale = kv_scale;
  return s;
}

int check_table(int32_t num_seqs, int32_t max_blocks_per_seq, int32_t block_size) {
  if (num_seqs < 0 || max_blocks_per_seq <= 0) return PA_ERR_INVALID_ARG;
  return static_cast<int64_t>(max_blocks_per_seq) * block_size > INT32_MAX ? PA_ERR_INVALID_ARG : PA_OK;
}

// Split runs: CTAs per SM when every context has the caller's largest length, and
// how many of a context's last partitions run by themselves at the end of the
// grid.  About one run per place, so that starts and merges are few: chosen
// contexts, which are equally long, 3 per SM over 16-bit caches and 4 over E4M3
// (65536 tokens of 8 heads, 128 channels, bf16: 64.8, 59.8, 59.2, 49.2 us with 9,
// 6, 4, 3).  Row-scaled ones 4 with 128 channels and, as a CTA's start is a
// larger share of its run, 6 with 64.  Measured over fifteen batches of 1 to 30
// contexts of 1000 to 131072 tokens, as the geometric mean of time over the
// bytes' floor: 1.58 with 9 and a fringe of 8; with 4 (6) and a fringe of 8, 6,
// 4, 3, 0: 1.51, 1.49, 1.46, 1.47, 1.48; with 3 (5) and 4: 1.55; 6 (6): 1.61.
int form_ctas_per_sm(const pa_cache_desc* c, bool row_scaled) {
  if (row_scaled) return c->head_dim == 64 ? 6 : 4;
  return c->kv_dtype == PA_FP8_E4M3 ? 4 : 3;
}
constexpr int kFormFringe = 4;

// What pa_decode_rows and pa_decode_selected check and launch alike.
struct FormArgs {
  void* out;
  const void* q;
  int32_t q_dtype, num_seqs, num_q_tokens, num_q_heads;
  const void* k_cache;
  const void* v_cache;
  const pa_cache_desc* cache;
  const int32_t* tables;
  int32_t max_blocks;
  const int32_t* lens;
  float scale, kv_scale;
  int32_t max_context_len, partition_size;
  void* workspace;
  size_t workspace_bytes;
};

int check_form(const FormArgs& a) {
  const pa_cache_desc* c = a.cache;
  int rc = check_table(a.num_seqs, a.max_blocks, c->block_size);
  if (rc) return rc;
  if (a.num_q_heads <= 0 || a.num_q_tokens < 1 || a.num_q_heads % c->num_kv_heads) return PA_ERR_INVALID_ARG;
  if (!is16(a.q_dtype) || (c->kv_dtype != PA_FP8_E4M3 && c->kv_dtype != a.q_dtype)) return PA_ERR_UNSUPPORTED;
  if (a.num_q_heads / c->num_kv_heads > 128 || a.num_q_tokens > pa::kMaxGroup) return PA_ERR_UNSUPPORTED;
  if (!std::isfinite(a.scale)) return PA_ERR_INVALID_ARG;
  if (a.partition_size < 0 || a.partition_size % pa::kTileTokens || a.max_context_len < 0) return PA_ERR_INVALID_ARG;
  if (a.num_seqs == 0) return PA_OK;
  if (!a.out || !a.q || !a.tables || !a.lens || !aligned16(a.out) || !aligned16(a.q)) return PA_ERR_INVALID_ARG;
  const int64_t np = a.partition_size ? pa::host::split_partitions(a.max_context_len, a.partition_size) : 1;
  const int64_t rows = static_cast<int64_t>(a.num_seqs) * a.num_q_tokens * a.num_q_heads;
  // CTAs: num_q_heads bounds the virtual heads, and a context's runs its partitions
  if (rows > INT32_MAX || static_cast<int64_t>(a.num_seqs) * a.num_q_heads * np > INT32_MAX) return PA_ERR_INVALID_ARG;
  if (a.partition_size) {
    const size_t need = pa_decode_multi_split_workspace_size(a.num_seqs, a.num_q_tokens, a.num_q_heads, c->head_dim,
                                                             a.max_context_len, a.partition_size);
    if (!a.workspace || a.workspace_bytes < need || !aligned16(a.workspace)) return PA_ERR_WORKSPACE;
  }
  return PA_OK;
}

// Sets everything but the form's own fields.
void form_params(const FormArgs& a, bool row_scaled, int* err, pa::DecodeParams& p) {
  const pa_cache_desc* c = a.cache;
  const int G = a.num_q_heads / c->num_kv_heads;
  p.out = a.out;
  p.q = a.q;
  p.block_tables = a.tables;
  p.context_lens = a.lens;
  p.err = err;
  p.num_blocks = c->num_blocks;
  p.S = a.num_seqs;
  p.Hq = a.num_q_heads;
  p.G = pa::host::heads_per_cta(G, a.num_q_tokens);
  p.head_div = G / p.G;
  p.Hkv = c->num_kv_heads * p.head_div;
  p.bs = c->block_size;
  p.maxB = a.max_blocks;
  p.qlen = a.num_q_tokens;
  p.q_dtype = a.q_dtype;
  p.Pmax = 1;
  p.parts_per_cta = 1;
  p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
  p.kv_scale = a.kv_scale;
  p.sms = pa::host::sms();
  p.cluster = 1;
  if (a.partition_size)
    pa::host::set_split(p, pa::host::split_partitions(a.max_context_len, a.partition_size), a.partition_size,
                        c->head_dim, a.workspace, form_ctas_per_sm(c, row_scaled), kFormFringe);
}

}  // namespace

extern "C" {

int pa_reshape_and_cache_rows(const void* key, const void* value, int32_t in_dtype, int32_t num_tokens, void* k_cache,
                              void* v_cache, float* k_scales, float* v_scales, const pa_cache_desc* cache,
                              const int64_t* slot_mapping, pa_stream_t stream) {
  int rc = pa::host::check_cache(cache, k_cache, v_cache);
  if (rc || (rc = check_row_scales(cache, k_scales, v_scales))) return rc;
  if (!is16(in_dtype)) return PA_ERR_UNSUPPORTED;
  if (num_tokens < 0) return PA_ERR_INVALID_ARG;
  if (num_tokens == 0) return PA_OK;
  if (!key || !value || !slot_mapping || !aligned16(key) || !aligned16(value)) return PA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(num_tokens) * cache->num_kv_heads > INT32_MAX * int64_t(16)) return PA_ERR_INVALID_ARG;
  int* err = error_word();
  if (!err) return PA_ERR_CUDA;
  pa::CacheRowsParams p{};
  p.key = key;
  p.value = value;
  p.T = num_tokens;
  p.bf16 = in_dtype == PA_BF16;
  p.sink = make_sink(k_cache, v_cache, k_scales, v_scales, cache, slot_mapping, 1.f, err);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return finish(pa::launch_cache_rows(p, st), st);
}

int pa_gather_blocks_rows(void* k_dst, void* v_dst, int32_t dst_dtype, const void* k_cache, const void* v_cache,
                          const float* k_scales, const float* v_scales, const pa_cache_desc* cache,
                          const int64_t* block_ids, int32_t num, pa_stream_t stream) {
  int rc = pa::host::check_cache(cache, k_cache, v_cache);
  if (rc || (rc = check_row_scales(cache, k_scales, v_scales))) return rc;
  if (!is16(dst_dtype)) return PA_ERR_UNSUPPORTED;
  if (num < 0) return PA_ERR_INVALID_ARG;
  if (num == 0) return PA_OK;
  if (!k_dst || !v_dst || !block_ids || !aligned16(k_dst) || !aligned16(v_dst)) return PA_ERR_INVALID_ARG;
  const int64_t rows = static_cast<int64_t>(cache->num_kv_heads) * cache->block_size;
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
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.ids = static_cast<const int64_t*>(ids);
  p.err = err;
  p.num_blocks = cache->num_blocks;
  p.n = num;
  p.rows = static_cast<int>(rows);
  p.D = cache->head_dim;
  p.bf16 = dst_dtype == PA_BF16;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return finish(pa::launch_gather_rows(p, st), st);
}

int pa_decode_rows(void* out, const void* q, int32_t q_dtype, int32_t num_seqs, int32_t num_q_tokens,
                   int32_t num_q_heads, const void* k_cache, const void* v_cache, const float* k_scales,
                   const float* v_scales, const pa_cache_desc* cache, const int32_t* block_tables,
                   int32_t max_blocks_per_seq, const int32_t* context_lens, float scale, int32_t max_context_len,
                   int32_t partition_size, void* workspace, size_t workspace_bytes, pa_stream_t stream) {
  int rc = pa::host::check_cache(cache, k_cache, v_cache);
  if (rc || (rc = check_row_scales(cache, k_scales, v_scales))) return rc;
  const FormArgs a{out, q, q_dtype, num_seqs, num_q_tokens, num_q_heads, k_cache, v_cache, cache, block_tables,
                   max_blocks_per_seq, context_lens, scale, 1.f, max_context_len, partition_size, workspace,
                   workspace_bytes};
  rc = check_form(a);
  if (rc || num_seqs == 0) return rc;
  int* err = error_word();
  if (!err) return PA_ERR_CUDA;
  CUtensorMap tk, tv;
  if ((rc = pa::host::make_cache_tensor_map(&tk, k_cache, cache)) ||
      (rc = pa::host::make_cache_tensor_map(&tv, v_cache, cache)))
    return rc;
  pa::DecodeParams p{};
  form_params(a, true, err, p);
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = pa::launch_decode_rows(p, tk, tv, cache->head_dim, st);
  if (e == cudaSuccess && partition_size) e = pa::launch_lse_merge(p, cache->head_dim, st);
  return finish(e, st);
}

int pa_norm_rope_cache(void* q_out, const void* q, int64_t q_stride, const void* key, int64_t key_stride,
                       const void* value, int64_t value_stride, int32_t dtype, int32_t num_tokens,
                       int32_t num_q_heads, const void* q_weight, const void* k_weight, float eps,
                       const int64_t* positions, const float* cos_sin, int64_t num_positions, int32_t rot_dim,
                       int32_t interleaved, void* k_cache, void* v_cache, float* k_scales, float* v_scales,
                       const pa_cache_desc* cache, const int64_t* slot_mapping, float kv_scale, pa_stream_t stream) {
  int rc = pa::host::check_cache(cache, k_cache, v_cache);
  if (rc) return rc;
  if (!is16(dtype) || (cache->kv_dtype != PA_FP8_E4M3 && cache->kv_dtype != dtype)) return PA_ERR_UNSUPPORTED;
  const bool rows = k_scales || v_scales;
  if (rows && (rc = check_row_scales(cache, k_scales, v_scales))) return rc;
  // 16-bit and row-scaled caches take a kv_scale of 1
  if ((rc = pa::host::check_kv_scale(rows ? dtype : cache->kv_dtype, kv_scale))) return rc;
  const int D = cache->head_dim;
  if (num_tokens < 0 || num_q_heads <= 0 || num_q_heads > 65535) return PA_ERR_INVALID_ARG;
  constexpr int64_t kMaxStride = int64_t(1) << 30;  // times num_tokens fits 64 bits
  for (const int64_t stride : {q_stride, key_stride, value_stride})
    if (stride < 0 || stride > kMaxStride || stride % 8) return PA_ERR_INVALID_ARG;
  if (!q_weight != !k_weight || !aligned16(q_weight) || !aligned16(k_weight)) return PA_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f) return PA_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim > D || rot_dim % 2 || (interleaved != 0 && interleaved != 1)) return PA_ERR_INVALID_ARG;
  if (!interleaved && rot_dim % 8) return PA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PA_OK;
  if (rot_dim > 0 && (!positions || !cos_sin || num_positions <= 0 || (reinterpret_cast<uintptr_t>(cos_sin) & 3)))
    return PA_ERR_INVALID_ARG;
  if (!q_out || !q || !key || !value || !slot_mapping || !aligned16(q_out) || !aligned16(q) || !aligned16(key) ||
      !aligned16(value))
    return PA_ERR_INVALID_ARG;
  const int64_t T = num_tokens, qw = static_cast<int64_t>(num_q_heads) * D;
  const int64_t kw = static_cast<int64_t>(cache->num_kv_heads) * D, out_bytes = T * qw * 2;
  const bool in_place = q_out == q && (q_stride == qw || T == 1);
  if ((!in_place && overlap(q_out, out_bytes, q, ((T - 1) * q_stride + qw) * 2)) ||
      overlap(q_out, out_bytes, key, ((T - 1) * key_stride + kw) * 2) ||
      overlap(q_out, out_bytes, value, ((T - 1) * value_stride + kw) * 2))
    return PA_ERR_INVALID_ARG;
  int* err = error_word();
  if (!err) return PA_ERR_CUDA;
  pa::NormRopeParams p{};
  p.q_out = q_out;
  p.q = q;
  p.key = key;
  p.value = value;
  p.q_stride = q_stride;
  p.key_stride = key_stride;
  p.value_stride = value_stride;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.num_positions = num_positions;
  p.T = num_tokens;
  p.Hq = num_q_heads;
  p.rot = rot_dim;
  p.interleaved = interleaved;
  p.bf16 = dtype == PA_BF16;
  p.sms = pa::host::sms();
  p.eps = eps;
  p.sink = make_sink(k_cache, v_cache, k_scales, v_scales, cache, slot_mapping, kv_scale, err);
  const int kind = rows ? pa::kSinkRows : (cache->kv_dtype == PA_FP8_E4M3 ? pa::kSinkTensor : pa::kSink16);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return finish(pa::launch_norm_rope(p, kind, st), st);
}

int pa_block_bounds(void* bounds, const void* k_cache, const pa_cache_desc* cache, const int32_t* block_tables,
                    int32_t max_blocks_per_seq, const int32_t* context_lens, int32_t num_seqs, int32_t num_new_tokens,
                    pa_stream_t stream) {
  int rc = pa::host::check_cache(cache, k_cache, k_cache);
  if (rc || (rc = check_table(num_seqs, max_blocks_per_seq, cache->block_size))) return rc;
  if (num_new_tokens < 1) return PA_ERR_INVALID_ARG;
  // more new tokens than the table holds are all of them
  const int bs = cache->block_size;
  const int new_tokens = std::min(num_new_tokens, max_blocks_per_seq * bs);
  const int touched =
      static_cast<int>(std::min<int64_t>((int64_t(new_tokens) + bs - 2) / bs + 1, max_blocks_per_seq));
  if (static_cast<int64_t>(num_seqs) * touched > INT32_MAX) return PA_ERR_INVALID_ARG;
  if (num_seqs == 0) return PA_OK;
  if (!bounds || !block_tables || !context_lens || !aligned16(bounds)) return PA_ERR_INVALID_ARG;
  int* err = error_word();
  if (!err) return PA_ERR_CUDA;
  pa::BoundsParams p{};
  p.bounds = bounds;
  p.k_cache = k_cache;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.err = err;
  p.num_blocks = cache->num_blocks;
  p.S = num_seqs;
  p.maxB = max_blocks_per_seq;
  p.Hkv = cache->num_kv_heads;
  p.D = cache->head_dim;
  p.bs = bs;
  p.num_new = new_tokens;
  p.touched = touched;
  p.kv_dtype = cache->kv_dtype;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return finish(pa::launch_block_bounds(p, st), st);
}

int pa_block_scores(float* scores, const void* q, int32_t q_dtype, int32_t num_seqs, int32_t num_q_heads,
                    const void* bounds, const pa_cache_desc* cache, const int32_t* block_tables,
                    int32_t max_blocks_per_seq, const int32_t* context_lens, pa_stream_t stream) {
  int rc = pa::host::check_cache(cache, bounds, bounds);
  if (rc || (rc = check_table(num_seqs, max_blocks_per_seq, cache->block_size))) return rc;
  if (!is16(q_dtype) || (cache->kv_dtype != PA_FP8_E4M3 && cache->kv_dtype != q_dtype)) return PA_ERR_UNSUPPORTED;
  if (num_q_heads <= 0 || num_q_heads % cache->num_kv_heads) return PA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(num_seqs) * cache->num_kv_heads * ((static_cast<int64_t>(max_blocks_per_seq) + 15) / 16) >
      INT32_MAX)
    return PA_ERR_INVALID_ARG;
  if (num_q_heads / cache->num_kv_heads > 128) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PA_OK;
  if (!scores || !q || !block_tables || !context_lens || !aligned16(q)) return PA_ERR_INVALID_ARG;
  int* err = error_word();
  if (!err) return PA_ERR_CUDA;
  pa::ScoresParams p{};
  p.scores = scores;
  p.q = q;
  p.bounds = bounds;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.err = err;
  p.num_blocks = cache->num_blocks;
  p.S = num_seqs;
  p.maxB = max_blocks_per_seq;
  p.Hq = num_q_heads;
  p.Hkv = cache->num_kv_heads;
  p.G = num_q_heads / cache->num_kv_heads;
  p.D = cache->head_dim;
  p.bs = cache->block_size;
  p.q_bf16 = q_dtype == PA_BF16;
  p.sms = pa::host::sms();
  p.kv_dtype = cache->kv_dtype;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return finish(pa::launch_block_scores(p, st), st);
}

int pa_select_blocks(int32_t* tables, int32_t* lens, int32_t num_selected, const float* scores,
                     const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
                     int32_t num_seqs, int32_t num_kv_heads, int32_t block_size, int32_t sink_blocks,
                     int32_t recent_blocks, pa_stream_t stream) {
  if (block_size != 8 && block_size != 16 && block_size != 32) return PA_ERR_UNSUPPORTED;
  const int rc = check_table(num_seqs, max_blocks_per_seq, block_size);
  if (rc) return rc;
  if (num_kv_heads <= 0 || num_kv_heads > 65535 || num_selected < 1 || sink_blocks < 0 || recent_blocks < 0 ||
      static_cast<int64_t>(sink_blocks) + recent_blocks > num_selected ||
      static_cast<int64_t>(num_selected) * block_size > INT32_MAX ||
      static_cast<int64_t>(num_seqs) * num_kv_heads > INT32_MAX)
    return PA_ERR_INVALID_ARG;
  if (num_seqs == 0) return PA_OK;
  if (!tables || !lens || !scores || !block_tables || !context_lens) return PA_ERR_INVALID_ARG;
  // a row's ids are written while other rows are read
  const int64_t rows = static_cast<int64_t>(num_seqs) * num_kv_heads, written = rows * num_selected * 4;
  if (overlap(tables, written, scores, rows * max_blocks_per_seq * 4) ||
      overlap(tables, written, block_tables, static_cast<int64_t>(num_seqs) * max_blocks_per_seq * 4))
    return PA_ERR_INVALID_ARG;
  int* err = error_word();
  if (!err) return PA_ERR_CUDA;
  pa::SelectParams p{};
  p.tables = tables;
  p.lens = lens;
  p.scores = scores;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.err = err;
  p.S = num_seqs;
  p.maxB = max_blocks_per_seq;
  p.Hkv = num_kv_heads;
  p.bs = block_size;
  p.n = num_selected;
  p.sink = sink_blocks;
  p.recent = recent_blocks;
  p.sms = pa::host::sms();
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return finish(pa::launch_select_blocks(p, st), st);
}

int pa_decode_selected(void* out, const void* q, int32_t q_dtype, int32_t num_seqs, int32_t num_q_heads,
                       const void* k_cache, const void* v_cache, const pa_cache_desc* cache, const int32_t* tables,
                       int32_t num_selected, const int32_t* lens, float scale, float kv_scale, int32_t partition_size,
                       void* workspace, size_t workspace_bytes, pa_stream_t stream) {
  int rc = pa::host::check_cache(cache, k_cache, v_cache);
  if (rc || (rc = pa::host::check_kv_scale(cache->kv_dtype, kv_scale))) return rc;
  if ((rc = check_table(num_seqs, num_selected, cache->block_size))) return rc;
  FormArgs a{out, q, q_dtype, num_seqs, 1, num_q_heads, k_cache, v_cache, cache, tables, num_selected, lens,
             scale, kv_scale, num_selected * cache->block_size, partition_size, workspace, workspace_bytes};
  rc = check_form(a);
  if (rc || num_seqs == 0) return rc;
  // The contexts are equally long, so in one pass they keep the GPU busy once
  // there are places enough, and a few are shared by clusters of 8 CTAs.  One
  // sequence of 8 heads, in one pass and in partitions of 64 and 512 tokens: 1024
  // tokens each 6.8, 8.1, 12.6 us, 4096: 11.2, 10.2, 12.6, 8192: 17.1, 12.3, 13.1.
  // From one context per SM on (8192 tokens each, bf16, one pass and the best of 64,
  // 256, 512): 168 contexts 96.7 and 100.8, 200: 126.8 and 117.0, 256: 150.4 and
  // 159.0, 400: 226.7 and 232.2.  E4M3 contexts would gain by partitions of 512 where
  // they fill less than half of the places: 168 74.7 and 58.4, 320: 137.3 and 106.5,
  // 152: 52.3 and 52.6, 400: 138.9 and 129.5.
  if (static_cast<int64_t>(num_seqs) * cache->num_kv_heads >= pa::host::sms() ||
      a.max_context_len <= 64 * pa::kTileTokens)
    a.partition_size = 0;
  int* err = error_word();
  if (!err) return PA_ERR_CUDA;
  CUtensorMap tk, tv;
  if ((rc = pa::host::make_cache_tensor_map(&tk, k_cache, cache)) ||
      (rc = pa::host::make_cache_tensor_map(&tv, v_cache, cache)))
    return rc;
  pa::DecodeParams p{};
  form_params(a, false, err, p);
  p.tab_heads = cache->num_kv_heads;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int D = cache->head_dim;
  cudaError_t e = cache->kv_dtype == PA_F16    ? pa::launch_decode_heads_f16(p, tk, tv, D, st)
                  : cache->kv_dtype == PA_BF16 ? pa::launch_decode_heads_bf16(p, tk, tv, D, st)
                                               : pa::launch_decode_heads_fp8(p, tk, tv, D, st);
  if (e == cudaSuccess && a.partition_size) e = pa::launch_lse_merge(p, D, st);
  return finish(e, st);
}

}  // extern "C"
