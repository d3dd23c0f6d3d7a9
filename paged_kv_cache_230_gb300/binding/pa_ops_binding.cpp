// Compiled marshalling of the cache-side operators (module _pa_ops, used by
// pagedattn.py).  A decode step calls several of them per layer, each a few
// microseconds on the GPU: checking ten tensors attribute by attribute from
// Python and converting twenty-five arguments costs more than that (14 us for
// norm_rope_cache against 4 here).  As the rest of the binding it only checks
// tensors and passes device pointers and the current stream to the C ABI; every
// function returns the library's status.
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pagedattn.h"

namespace {

struct Refused {};  // a Python error is set

[[noreturn]] void refuse(PyObject* type, const char* format, const char* name) {
  PyErr_Format(type, format, name);
  throw Refused();
}

bool is_none(PyObject* o) { return o == Py_None; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_CheckExact(o) && !THPVariable_Check(o)) refuse(PyExc_ValueError, "%s must be a CUDA tensor", name);
  return THPVariable_Unpack(o);
}

int32_t i32(PyObject* o, const char* name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_ValueError, "%s is out of range", name);
  return static_cast<int32_t>(v);
}

int32_t size32(int64_t n, const char* name) {
  if (n > INT32_MAX) refuse(PyExc_ValueError, "%s is too large", name);
  return static_cast<int32_t>(n);
}

float f32(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return static_cast<float>(v);
}

bool is_half(at::ScalarType t) { return t == at::kHalf || t == at::kBFloat16; }
bool is_e4m3(at::ScalarType t) { return t == at::kByte || t == at::kFloat8_e4m3fn; }

int32_t dtype_code(at::ScalarType t) {
  if (t == at::kHalf) return PA_F16;
  if (t == at::kBFloat16) return PA_BF16;
  if (is_e4m3(t)) return PA_FP8_E4M3;
  refuse(PyExc_TypeError, "%s has an unsupported dtype", "the cache");
}

// This type and shape (strides apart).
void want_type(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape) {
  if (t.scalar_type() != type) refuse(PyExc_TypeError, "%s has another dtype than the call takes", name);
  if (t.sizes() != shape) refuse(PyExc_ValueError, "%s has another shape than the other tensors ask for", name);
}

// A tensor of device `dev` with this type and shape.
void want_like(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, int dev) {
  if (!t.is_cuda() || t.get_device() != dev)
    refuse(PyExc_ValueError, "%s must be a CUDA tensor on the device of the other tensors", name);
  want_type(t, name, type, shape);
}

void want_dense(const at::Tensor& t, const char* name) {
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
}

template <class T = void>
T* want(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, int dev) {
  const at::Tensor& t = tensor(o, name);
  want_like(t, name, type, shape, dev);
  want_dense(t, name);
  return static_cast<T*>(t.data_ptr());
}

// The same for a buffer that may be pinned host memory, which kernels reach through its mapping.
void* want_buffer(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, int dev) {
  const at::Tensor& t = tensor(o, name);
  if (t.is_cuda()) return want(o, name, type, shape, dev);
  if (!t.is_cpu() || !t.is_pinned()) refuse(PyExc_ValueError, "%s must be a CUDA tensor or pinned host memory", name);
  want_type(t, name, type, shape);
  want_dense(t, name);
  return t.data_ptr();
}

const at::Tensor& with_dims(PyObject* o, const char* name, int64_t dims) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != dims) refuse(PyExc_ValueError, "%s has the wrong number of dimensions", name);
  return t;
}

struct Pool {
  int dev;
  at::ScalarType type;
  pa_cache_desc desc;
  at::IntArrayRef shape;
  void* k;
  void* v;
};

Pool pool(PyObject* k, PyObject* v, const char* k_name = "k_cache", const char* v_name = "v_cache") {
  const at::Tensor& t = with_dims(k, k_name, 4);
  if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", k_name);
  Pool p;
  p.dev = t.get_device();
  p.type = t.scalar_type();
  p.shape = t.sizes();
  p.desc = {t.size(0), size32(t.size(2), k_name), size32(t.size(1), k_name), size32(t.size(3), k_name),
            dtype_code(p.type)};
  p.k = want(k, k_name, p.type, p.shape, p.dev);
  p.v = v == k ? p.k : want(v, v_name, p.type, p.shape, p.dev);
  return p;
}

struct Scales {
  float* k = nullptr;
  float* v = nullptr;
};

Scales scales(const Pool& p, PyObject* k, PyObject* v) {
  if (!is_e4m3(p.type)) refuse(PyExc_TypeError, "%s belong to E4M3 caches", "row scales");
  return {want<float>(k, "k_scales", at::kFloat, p.shape.slice(0, 3), p.dev),
          want<float>(v, "v_scales", at::kFloat, p.shape.slice(0, 3), p.dev)};
}

at::ScalarType half_type(const at::Tensor& t, const char* name) {
  if (!is_half(t.scalar_type())) refuse(PyExc_TypeError, "%s must be float16 or bfloat16", name);
  return t.scalar_type();
}

struct Workspace {
  void* ptr = nullptr;
  size_t bytes = 0;
};

Workspace workspace(PyObject* o, int dev) {
  if (is_none(o)) return {};
  const at::Tensor& t = tensor(o, "workspace");
  if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
    refuse(PyExc_ValueError, "%s must be a contiguous CUDA tensor on the cache's device", "workspace");
  return {t.data_ptr(), t.nbytes()};
}

// The library call, on the current stream of `dev`, without the interpreter lock.
template <class Call>
PyObject* launch(int dev, Call call) {
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  const pa_stream_t st = reinterpret_cast<pa_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream());
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = call(st);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

using Args = PyObject* const*;

PyObject* reshape_and_cache_rows(Args a) {  // key, value, k_cache, v_cache, k_scales, v_scales, slot_mapping
  const Pool p = pool(a[2], a[3]);
  const Scales s = scales(p, a[4], a[5]);
  const at::Tensor& key = with_dims(a[0], "key", 3);
  const at::ScalarType type = half_type(key, "key");
  const int64_t T = key.size(0), shape[] = {T, p.shape[1], p.shape[3]};
  const void* k = want(a[0], "key", type, shape, p.dev);
  const void* v = want(a[1], "value", type, shape, p.dev);
  const int64_t* slots = want<int64_t>(a[6], "slot_mapping", at::kLong, {T}, p.dev);
  const int32_t T32 = size32(T, "key");
  return launch(p.dev, [&](pa_stream_t st) {
    return pa_reshape_and_cache_rows(k, v, dtype_code(type), T32, p.k, p.v, s.k, s.v, &p.desc, slots, st);
  });
}

PyObject* gather_blocks_rows(Args a) {  // k_dst, v_dst, k_cache, v_cache, k_scales, v_scales, ids
  const Pool p = pool(a[2], a[3]);
  const Scales s = scales(p, a[4], a[5]);
  const at::Tensor& dst = with_dims(a[0], "k_dst", 4);
  const at::ScalarType type = half_type(dst, "k_dst");
  const int64_t n = dst.size(0), shape[] = {n, p.shape[1], p.shape[2], p.shape[3]};
  void* k = want_buffer(a[0], "k_dst", type, shape, p.dev);
  void* v = want_buffer(a[1], "v_dst", type, shape, p.dev);
  const int64_t* ids = want<int64_t>(a[6], "ids", at::kLong, {n}, p.dev);
  const int32_t n32 = size32(n, "k_dst");
  return launch(p.dev, [&](pa_stream_t st) {
    return pa_gather_blocks_rows(k, v, dtype_code(type), p.k, p.v, s.k, s.v, &p.desc, ids, n32, st);
  });
}

PyObject* decode_rows(Args a) {  // out, q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, scale,
                                 // max_context_len, partition_size, workspace
  const Pool p = pool(a[2], a[3]);
  const Scales s = scales(p, a[4], a[5]);
  const at::Tensor& q = tensor(a[1], "q");
  const at::ScalarType type = half_type(q, "q");
  if (q.dim() != 3 && q.dim() != 4) refuse(PyExc_ValueError, "%s must have 3 or 4 dims", "q");
  const int64_t S = q.size(0), k = q.dim() == 4 ? q.size(1) : 1, Hq = q.size(-2);
  const void* qp = want(a[1], "q", type, q.sizes(), p.dev);
  if (q.size(-1) != p.shape[3]) refuse(PyExc_ValueError, "%s has another head_dim than the cache", "q");
  void* out = want(a[0], "out", type, q.sizes(), p.dev);
  const int64_t maxB = with_dims(a[6], "block_tables", 2).size(1);
  const int32_t* bt = want<int32_t>(a[6], "block_tables", at::kInt, {S, maxB}, p.dev);
  const int32_t* cl = want<int32_t>(a[7], "context_lens", at::kInt, {S}, p.dev);
  const float scale = f32(a[8]);
  const int32_t most = i32(a[9], "max_context_len"), P = i32(a[10], "partition_size");
  const Workspace ws = workspace(a[11], p.dev);
  const int32_t S32 = size32(S, "q"), k32 = size32(k, "q"), H32 = size32(Hq, "q"), B32 = size32(maxB, "block_tables");
  return launch(p.dev, [&](pa_stream_t st) {
    return pa_decode_rows(out, qp, dtype_code(type), S32, k32, H32, p.k, p.v, s.k, s.v, &p.desc, bt, B32, cl, scale,
                          most, P, ws.ptr, ws.bytes, st);
  });
}

// Pointer and token stride of [T, H, D] rows whose heads are contiguous within a token.
const void* token_rows(PyObject* o, const char* name, at::ScalarType type, int64_t T, int64_t H, int64_t D, int dev,
                       int64_t* stride) {
  const at::Tensor& t = tensor(o, name);
  const int64_t shape[] = {T, H, D};
  want_like(t, name, type, shape, dev);
  if ((t.stride(2) != 1 && D > 1) || (t.stride(1) != D && H > 1))
    refuse(PyExc_ValueError, "the heads of %s must be contiguous within a token", name);
  *stride = T > 1 ? t.stride(0) : H * D;
  return t.data_ptr();
}

PyObject* norm_rope_cache(Args a) {  // q_out, q, key, value, positions, cos_sin, k_cache, v_cache, slot_mapping,
                                     // q_weight, k_weight, eps, interleaved, kv_scale, k_scales, v_scales
  const Pool p = pool(a[6], a[7]);
  const at::Tensor& q = with_dims(a[1], "q", 3);
  const at::ScalarType type = half_type(q, "q");
  const int64_t T = q.size(0), Hq = q.size(1), Hkv = p.shape[1], D = p.shape[3];
  int64_t qs, ks, vs;
  const void* qp = token_rows(a[1], "q", type, T, Hq, D, p.dev, &qs);
  const void* kp = token_rows(a[2], "key", type, T, Hkv, D, p.dev, &ks);
  const void* vp = token_rows(a[3], "value", type, T, Hkv, D, p.dev, &vs);
  void* out = want(a[0], "q_out", type, q.sizes(), p.dev);
  const int64_t* slots = want<int64_t>(a[8], "slot_mapping", at::kLong, {T}, p.dev);
  const void* qw = nullptr;
  const void* kw = nullptr;
  if (is_none(a[9]) != is_none(a[10])) refuse(PyExc_ValueError, "%s come together", "q_weight and k_weight");
  if (!is_none(a[9])) {
    qw = want(a[9], "q_weight", type, {D}, p.dev);
    kw = want(a[10], "k_weight", type, {D}, p.dev);
  }
  const int64_t* pos = nullptr;
  const float* table = nullptr;
  int64_t rows = 0;
  int32_t rot = 0;
  if (!is_none(a[5])) {
    const at::Tensor& t = with_dims(a[5], "cos_sin", 2);
    table = want<float>(a[5], "cos_sin", at::kFloat, t.sizes(), p.dev);
    pos = want<int64_t>(a[4], "positions", at::kLong, {T}, p.dev);
    rows = t.size(0);
    rot = size32(t.size(1), "cos_sin");
  }
  Scales s;
  if (is_none(a[14]) != is_none(a[15])) refuse(PyExc_ValueError, "%s come together", "k_scales and v_scales");
  if (!is_none(a[14])) s = scales(p, a[14], a[15]);
  const float eps = f32(a[11]), kv_scale = f32(a[13]);
  const int inter = PyObject_IsTrue(a[12]);
  if (inter < 0) throw Refused();
  const int32_t T32 = size32(T, "q"), H32 = size32(Hq, "q");
  return launch(p.dev, [&](pa_stream_t st) {
    return pa_norm_rope_cache(out, qp, qs, kp, ks, vp, vs, dtype_code(type), T32, H32, qw, kw, eps, pos, table, rows,
                              rot, inter, p.k, p.v, s.k, s.v, &p.desc, slots, kv_scale, st);
  });
}

PyObject* block_bounds(Args a) {  // bounds, k_cache, block_tables, context_lens, num_new_tokens
  const Pool p = pool(a[1], a[1]);
  const int64_t shape[] = {p.shape[0], p.shape[1], 2, p.shape[3]};
  void* bounds = want(a[0], "bounds", p.type, shape, p.dev);
  const at::Tensor& bt = with_dims(a[2], "block_tables", 2);
  const int32_t* table = want<int32_t>(a[2], "block_tables", at::kInt, bt.sizes(), p.dev);
  const int32_t* cl = want<int32_t>(a[3], "context_lens", at::kInt, {bt.size(0)}, p.dev);
  const int32_t n = i32(a[4], "num_new_tokens"), S = size32(bt.size(0), "block_tables"),
                maxB = size32(bt.size(1), "block_tables");
  return launch(p.dev, [&](pa_stream_t st) { return pa_block_bounds(bounds, p.k, &p.desc, table, maxB, cl, S, n, st); });
}

PyObject* block_scores(Args a) {  // scores, q, bounds, block_tables, context_lens, block_size
  Pool p = pool(a[2], a[2], "bounds", "bounds");
  if (p.shape[2] != 2) refuse(PyExc_ValueError, "%s must be [num_blocks, num_kv_heads, 2, head_dim]", "bounds");
  p.desc.block_size = i32(a[5], "block_size");
  const at::Tensor& q = with_dims(a[1], "q", 3);
  const at::ScalarType type = half_type(q, "q");
  const at::Tensor& bt = with_dims(a[3], "block_tables", 2);
  const int64_t S = bt.size(0), maxB = bt.size(1), Hq = q.size(1);
  const void* qp = want(a[1], "q", type, {S, Hq, p.shape[3]}, p.dev);
  const int32_t* table = want<int32_t>(a[3], "block_tables", at::kInt, {S, maxB}, p.dev);
  const int32_t* cl = want<int32_t>(a[4], "context_lens", at::kInt, {S}, p.dev);
  float* scores = want<float>(a[0], "scores", at::kFloat, {S, p.shape[1], maxB}, p.dev);
  const int32_t S32 = size32(S, "q"), H32 = size32(Hq, "q"), B32 = size32(maxB, "block_tables");
  return launch(p.dev, [&](pa_stream_t st) {
    return pa_block_scores(scores, qp, dtype_code(type), S32, H32, p.k, &p.desc, table, B32, cl, st);
  });
}

PyObject* select_blocks(Args a) {  // tables, lens, scores, block_tables, context_lens, block_size, sink, recent
  const at::Tensor& sc = with_dims(a[2], "scores", 3);
  if (!sc.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", "scores");
  const int dev = sc.get_device();
  const int64_t S = sc.size(0), H = sc.size(1), maxB = sc.size(2);
  const float* scores = want<float>(a[2], "scores", at::kFloat, sc.sizes(), dev);
  const int32_t* bt = want<int32_t>(a[3], "block_tables", at::kInt, {S, maxB}, dev);
  const int32_t* cl = want<int32_t>(a[4], "context_lens", at::kInt, {S}, dev);
  const int64_t n = with_dims(a[0], "tables", 3).size(2);
  int32_t* tables = want<int32_t>(a[0], "tables", at::kInt, {S, H, n}, dev);
  int32_t* lens = want<int32_t>(a[1], "lens", at::kInt, {S, H}, dev);
  const int32_t bs = i32(a[5], "block_size"), sink = i32(a[6], "sink_blocks"), recent = i32(a[7], "recent_blocks");
  const int32_t S32 = size32(S, "scores"), H32 = size32(H, "scores"), B32 = size32(maxB, "scores"),
                n32 = size32(n, "tables");
  return launch(dev, [&](pa_stream_t st) {
    return pa_select_blocks(tables, lens, n32, scores, bt, B32, cl, S32, H32, bs, sink, recent, st);
  });
}

PyObject* decode_selected(Args a) {  // out, q, k_cache, v_cache, tables, lens, scale, kv_scale, partition_size,
                                     // workspace
  const Pool p = pool(a[2], a[3]);
  const at::Tensor& q = with_dims(a[1], "q", 3);
  const at::ScalarType type = half_type(q, "q");
  const int64_t S = q.size(0), Hq = q.size(1), n = with_dims(a[4], "tables", 3).size(2);
  const int64_t shape[] = {S, Hq, p.shape[3]};
  const void* qp = want(a[1], "q", type, shape, p.dev);
  void* out = want(a[0], "out", type, shape, p.dev);
  const int32_t* tables = want<int32_t>(a[4], "tables", at::kInt, {S, p.shape[1], n}, p.dev);
  const int32_t* lens = want<int32_t>(a[5], "lens", at::kInt, {S, p.shape[1]}, p.dev);
  const float scale = f32(a[6]), kv_scale = f32(a[7]);
  const int32_t P = i32(a[8], "partition_size");
  const Workspace ws = workspace(a[9], p.dev);
  const int32_t S32 = size32(S, "q"), H32 = size32(Hq, "q"), n32 = size32(n, "tables");
  return launch(p.dev, [&](pa_stream_t st) {
    return pa_decode_selected(out, qp, dtype_code(type), S32, H32, p.k, p.v, &p.desc, tables, n32, lens, scale,
                              kv_scale, P, ws.ptr, ws.bytes, st);
  });
}

template <PyObject* (*Fn)(Args), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return Fn(args);
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

#define PA_ENTRY(name, n) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<name, n>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {PA_ENTRY(reshape_and_cache_rows, 7),
                         PA_ENTRY(gather_blocks_rows, 7),
                         PA_ENTRY(decode_rows, 12),
                         PA_ENTRY(norm_rope_cache, 16),
                         PA_ENTRY(block_bounds, 5),
                         PA_ENTRY(block_scores, 6),
                         PA_ENTRY(select_blocks, 8),
                         PA_ENTRY(decode_selected, 10),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pa_ops", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__pa_ops(void) { return PyModule_Create(&module); }
