// Python module of the streaming entry points: tensor checks and argument
// marshalling in C++.  A single-token call takes a few microseconds on the
// GPU; marshalling it through ctypes took 15 to 45 us of host time, this takes
// 2 to 4.  The structures stay the ctypes ones of the package (filled and read
// through the buffer protocol), so both sides see the layout of svsa.h.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Stream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <string>

#include "svsa.h"

namespace {

struct Fail {};                                  // a Python exception is set

[[noreturn]] void fail(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw Fail{};
}

std::string text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

// A tensor argument; null for None where that is allowed.
const at::Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
  if (o == Py_None) {
    if (optional) return nullptr;
    fail(std::string(name) + " is None");
  }
  if (!THPVariable_Check(o)) fail(std::string(name) + ": expected a tensor");
  return &THPVariable_Unpack(o);
}

std::string got(const at::Tensor& t) {
  return std::string(c10::toString(t.scalar_type())) + " " + text(t.sizes()) + " strides " + text(t.strides()) +
         " on device " + std::to_string(t.get_device());
}

bool same(at::IntArrayRef a, std::initializer_list<int64_t> b) {
  return a.size() == b.size() && std::equal(a.begin(), a.end(), b.begin());
}

// The address of a contiguous tensor of this type, shape and device.
void* dense(const at::Tensor* t, at::ScalarType type, std::initializer_list<int64_t> shape, int device, const char* name) {
  if (t == nullptr) return nullptr;
  if (t->scalar_type() != type || !same(t->sizes(), shape) || !t->is_contiguous() || t->get_device() != device)
    fail(std::string(name) + ": expected a contiguous " + c10::toString(type) + " tensor " +
         text(at::IntArrayRef(shape.begin(), shape.size())) + " on device " + std::to_string(device) + ", got " + got(*t));
  return t->data_ptr();
}

// The address of a view [B, heads, N, d] with these strides (where a dimension is not of size 1) and a contiguous last
// dimension.
void* view(const at::Tensor* t, at::ScalarType type, std::initializer_list<int64_t> shape, const int64_t stride[3],
           int device, const char* name) {
  if (t == nullptr) return nullptr;
  bool fits = t->scalar_type() == type && same(t->sizes(), shape) && t->get_device() == device && t->stride(3) == 1;
  for (int e = 0; fits && e < 3; ++e) fits = t->size(e) == 1 || t->stride(e) == stride[e];
  if (!fits)
    fail(std::string(name) + ": expected " + c10::toString(type) + " " + text(at::IntArrayRef(shape.begin(), shape.size())) +
         " as in the parameters, with a contiguous last dimension, on device " + std::to_string(device) + ", got " + got(*t));
  return t->data_ptr();
}

// An N-dimensional tensor with a contiguous last dimension.
void four(const at::Tensor& t, const char* name) {
  if (t.dim() != 4 || t.stride(3) != 1) fail(std::string(name) + ": expected [B, heads, tokens, d] with a contiguous last dimension, got " + got(t));
}

int dtype_of(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return SVSA_BF16;
  if (t.scalar_type() == at::kHalf) return SVSA_F16;
  fail(std::string(name) + ": expected bfloat16 or float16, got " + got(t));
}
at::ScalarType type_of(int dtype) { return dtype == SVSA_F16 ? at::kHalf : at::kBFloat16; }

// A workspace and the bytes of it that the call may use.
void* workspace(const at::Tensor* ws, int64_t bytes, int device) {
  if (ws == nullptr) return nullptr;
  if (ws->get_device() != device || !ws->is_contiguous() || bytes < 0 || (size_t)bytes > ws->nbytes())
    fail("ws: expected a contiguous tensor of at least ws_bytes=" + std::to_string(bytes) + " bytes on device " +
         std::to_string(device) + ", got " + got(*ws));
  return ws->data_ptr();
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Fail{};
  return v;
}
int32_t int32_of(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX) fail(std::string(name) + "=" + std::to_string(v) + " does not fit 32 bits");
  return (int32_t)v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Fail{};
  return v != 0;
}

// The bytes of a ctypes structure.
template <typename T>
class Struct {
 public:
  Struct(PyObject* o, bool writable, const char* name) {
    if (PyObject_GetBuffer(o, &buf_, writable ? PyBUF_WRITABLE : PyBUF_SIMPLE) != 0) throw Fail{};
    if (buf_.len != (Py_ssize_t)sizeof(T)) {
      PyBuffer_Release(&buf_);
      fail(std::string(name) + ": not the parameters of this call");
    }
  }
  ~Struct() { PyBuffer_Release(&buf_); }
  Struct(const Struct&) = delete;
  Struct& operator=(const Struct&) = delete;
  T* operator->() const { return static_cast<T*>(buf_.buf); }
  T& operator*() const { return *static_cast<T*>(buf_.buf); }

 private:
  Py_buffer buf_;
};

PyObject* g_types[4];                            // NormRopeParams, Cache, CacheTokens, CacheQuery
PyObject* g_device;                              // "device"

// A new structure of g_types[which] holding `value`.
template <typename T>
PyObject* make(int which, const T& value) {
  PyObject* o = PyObject_CallNoArgs(g_types[which]);
  if (o == nullptr) throw Fail{};
  try {
    Struct<T> s(o, true, "structure");
    *s = value;
  } catch (...) {
    Py_DECREF(o);
    throw;
  }
  return o;
}

// Device of the call and its stream: `stream` or the device's current one.
class Launch {
 public:
  Launch(int device, PyObject* stream) {
    if (device < 0) fail("the tensors must be on a CUDA device");
    if (stream == Py_None) {
      handle_ = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    } else {
      PyObject* h = PyObject_GetAttrString(stream, "cuda_stream");
      if (h == nullptr) throw Fail{};
      handle_ = PyLong_AsVoidPtr(h);
      Py_DECREF(h);
      if (PyErr_Occurred()) throw Fail{};
    }
    guard_.emplace((c10::DeviceIndex)device);
  }
  void* stream() const { return handle_; }

 private:
  void* handle_;
  std::optional<c10::cuda::CUDAGuard> guard_;
};

template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Fail&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    throw Fail{};
  }
}

// norm_rope_params(q, k, cos, pos, rows, pairs, halves, eps)
PyObject* norm_rope_params(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() {
    count(n, 8);
    const at::Tensor& q = *tensor(a[0], "q");
    const at::Tensor *k = tensor(a[1], "k", true), *cos = tensor(a[2], "cos", true), *pos = tensor(a[3], "pos", true);
    four(q, "q");
    svsa_norm_rope p{};
    p.dtype = dtype_of(q, "q");
    p.B = int32_of(q.size(0), "B");
    p.heads_q = int32_of(q.size(1), "heads");
    p.N = int32_of(q.size(2), "tokens");
    p.d = int32_of(q.size(3), "d");
    for (int e = 0; e < 3; ++e) p.q_stride[e] = q.stride(e);
    if (k) {
      four(*k, "k");
      if (k->scalar_type() != q.scalar_type() || k->size(0) != q.size(0) || k->size(2) != q.size(2) || k->size(3) != q.size(3))
        fail("k: expected q's type, batch, tokens and head dim, got " + got(*k));
      p.heads_k = int32_of(k->size(1), "heads");
      for (int e = 0; e < 3; ++e) p.k_stride[e] = k->stride(e);
    }
    p.rows = a[4] == Py_None ? p.N : int32_of(integer(a[4]), "rows");
    PyObject* pairs = PySequence_Fast(a[5], "pairs: expected a sequence");
    if (pairs == nullptr) throw Fail{};
    const Py_ssize_t axes = PySequence_Fast_GET_SIZE(pairs);
    int64_t each[3] = {0, 0, 0};
    for (Py_ssize_t e = 0; e < axes && e < 3; ++e) each[e] = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(pairs, e));
    Py_DECREF(pairs);
    if (PyErr_Occurred()) throw Fail{};
    if (axes > 3) fail("pairs: at most 3 position axes");
    for (int e = 0; e < 3; ++e) p.pairs[e] = int32_of(each[e], "pairs");
    p.axes = (int32_t)axes;
    if (axes) {
      if (!pos || !cos) fail("to rotate, cos, sin and pos are needed");
      if (pos->dim() != 3 || cos->dim() != 2) fail("pos: expected [B or 1, N, axes]; cos: [rows, d / 2]");
      p.pos_stride = pos->size(0) == p.B && p.B > 1 ? (int64_t)p.N * axes : 0;
      p.table_rows = int32_of(cos->size(0), "table rows");
    }
    p.pairing = truth(a[6]) ? SVSA_PAIR_HALVES : SVSA_PAIR_ADJACENT;
    p.eps = (float)PyFloat_AsDouble(a[7]);
    if (PyErr_Occurred()) throw Fail{};
    return make(0, p);
  });
}

// The inputs that the forward and the backward share, from a[0] on: q k wq wk cos sin pos map.
struct RopeInputs {
  const at::Tensor *q, *k;
  void *pq, *pk, *wq, *wk, *cos = nullptr, *sin = nullptr, *pos = nullptr, *map;
  int device;
  at::ScalarType type;
};
RopeInputs rope_inputs(PyObject* const* a, const svsa_norm_rope& p, int64_t n_map) {
  RopeInputs r;
  r.q = tensor(a[0], "q");
  r.k = tensor(a[1], "k", true);
  r.device = r.q->get_device();
  r.type = type_of(p.dtype);
  if ((r.k == nullptr) != (p.heads_k == 0)) fail("k does not fit the parameters");
  r.pq = view(r.q, r.type, {p.B, p.heads_q, p.N, p.d}, p.q_stride, r.device, "q");
  r.pk = view(r.k, r.type, {p.B, p.heads_k, p.N, p.d}, p.k_stride, r.device, "k");
  r.wq = dense(tensor(a[2], "wq", true), at::kFloat, {p.d}, r.device, "wq");
  r.wk = dense(tensor(a[3], "wk", true), at::kFloat, {p.d}, r.device, "wk");
  if (p.axes) {
    r.cos = dense(tensor(a[4], "cos"), at::kFloat, {p.table_rows, p.d / 2}, r.device, "cos");
    r.sin = dense(tensor(a[5], "sin"), at::kFloat, {p.table_rows, p.d / 2}, r.device, "sin");
    r.pos = dense(tensor(a[6], "pos"), at::kInt, {p.pos_stride ? p.B : 1, p.N, p.axes}, r.device, "pos");
  }
  r.map = dense(tensor(a[7], "token map", true), at::kInt, {n_map}, r.device, "token map");
  return r;
}

// qk_norm_rope(q, k, wq, wk, cos, sin, pos, perm, yq, yk, params, stream)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() {
    count(n, 12);
    Struct<svsa_norm_rope> p(a[10], false, "p");
    const RopeInputs r = rope_inputs(a, *p, p->rows);
    void* yq = dense(tensor(a[8], "yq"), r.type, {p->B, p->heads_q, p->rows, p->d}, r.device, "yq");
    void* yk = dense(tensor(a[9], "yk", true), r.type, {p->B, p->heads_k, p->rows, p->d}, r.device, "yk");
    Launch l(r.device, a[11]);
    return PyLong_FromLong(svsa_qk_norm_rope(r.pq, r.pk, (float*)r.wq, (float*)r.wk, (float*)r.cos, (float*)r.sin,
                                             (int32_t*)r.pos, (int32_t*)r.map, yq, yk, &*p, l.stream()));
  });
}

// qk_norm_rope_bwd(dyq, dyk, q, k, wq, wk, cos, sin, pos, iperm, dq, dk, dwq, dwk, params, ws, ws_bytes, stream)
PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() {
    count(n, 18);
    Struct<svsa_norm_rope> given(a[14], false, "p");
    svsa_norm_rope p = *given;
    const RopeInputs r = rope_inputs(a + 2, p, p.N);
    void* dyq = dense(tensor(a[0], "dyq"), r.type, {p.B, p.heads_q, p.rows, p.d}, r.device, "dyq");
    void* dyk = dense(tensor(a[1], "dyk", true), r.type, {p.B, p.heads_k, p.rows, p.d}, r.device, "dyk");
    const at::Tensor *dq = tensor(a[10], "dq"), *dk = tensor(a[11], "dk", r.k == nullptr);
    four(*dq, "dq");
    for (int e = 0; e < 3; ++e) p.dq_stride[e] = dq->stride(e);
    if (r.k) {
      four(*dk, "dk");
      for (int e = 0; e < 3; ++e) p.dk_stride[e] = dk->stride(e);
    }
    void* pdq = view(dq, r.type, {p.B, p.heads_q, p.N, p.d}, p.dq_stride, r.device, "dq");
    void* pdk = r.k ? view(dk, r.type, {p.B, p.heads_k, p.N, p.d}, p.dk_stride, r.device, "dk") : nullptr;
    void* dwq = dense(tensor(a[12], "dwq", true), at::kFloat, {p.d}, r.device, "dwq");
    void* dwk = dense(tensor(a[13], "dwk", true), at::kFloat, {p.d}, r.device, "dwk");
    const int64_t bytes = integer(a[16]);
    void* ws = workspace(tensor(a[15], "ws", true), bytes, r.device);
    Launch l(r.device, a[17]);
    return PyLong_FromLong(svsa_qk_norm_rope_bwd(dyq, dyk, r.pq, r.pk, (float*)r.wq, (float*)r.wk, (float*)r.cos,
                                                 (float*)r.sin, (int32_t*)r.pos, (int32_t*)r.map, pdq, pdk, (float*)dwq,
                                                 (float*)dwk, &p, ws, (size_t)bytes, l.stream()));
  });
}

// block_cache(k, v, k_scale, v_scale, table, length, mean, mean_scale)
PyObject* block_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() {
    count(n, 8);
    const at::Tensor& k = *tensor(a[0], "k");
    const at::Tensor& table = *tensor(a[4], "table");
    const at::ScalarType type = k.scalar_type();
    if ((type != at::kFloat8_e4m3fn && type != at::kChar) || k.dim() != 4 || k.size(2) != 64)
      fail("k: expected float8_e4m3fn or int8 codes [n_pages, heads, 64, d], got " + got(k));
    if (table.dim() != 2) fail("table: expected [B, max_blocks], got " + got(table));
    const int dev = k.get_device();
    const int64_t pages = k.size(0), heads = k.size(1), d = k.size(3), B = table.size(0), width = table.size(1);
    svsa_cache c{};
    c.k = dense(&k, type, {pages, heads, 64, d}, dev, "k");
    c.v = dense(tensor(a[1], "v"), type, {pages, heads, 64, d}, dev, "v");
    c.k_scale = (float*)dense(tensor(a[2], "k_scale"), at::kFloat, {pages, heads}, dev, "k_scale");
    c.v_scale = (float*)dense(tensor(a[3], "v_scale"), at::kFloat, {pages, heads}, dev, "v_scale");
    c.table = (int32_t*)dense(&table, at::kInt, {B, width}, dev, "table");
    c.len = (int32_t*)dense(tensor(a[5], "length"), at::kInt, {B}, dev, "length");
    c.mean = (int8_t*)dense(tensor(a[6], "mean", true), at::kChar, {pages, heads, d}, dev, "mean");
    c.mean_scale = (float*)dense(tensor(a[7], "mean_scale", true), at::kFloat, {pages, heads}, dev, "mean_scale");
    c.B = int32_of(B, "B");
    c.heads = int32_of(heads, "heads");
    c.d = int32_of(d, "d");
    c.code = type == at::kChar ? SVSA_CODE_I8 : SVSA_CODE_E4M3;
    c.n_pages = int32_of(pages, "n_pages");
    c.max_blocks = int32_of(width, "max_blocks");
    PyObject* o = make(1, c);
    PyObject* index = PyLong_FromLong(dev);
    const int bad = index == nullptr || PyObject_SetAttr(o, g_device, index) != 0;
    Py_XDECREF(index);
    if (bad) {
      Py_DECREF(o);
      throw Fail{};
    }
    return o;
  });
}

int device_of(PyObject* cache) {
  PyObject* o = PyObject_GetAttr(cache, g_device);
  if (o == nullptr) throw Fail{};
  const long v = PyLong_AsLong(o);
  Py_DECREF(o);
  if (v == -1 && PyErr_Occurred()) throw Fail{};
  return (int)v;
}

// cache_tokens(k, v)
PyObject* cache_tokens(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() {
    count(n, 2);
    const at::Tensor &k = *tensor(a[0], "k"), &v = *tensor(a[1], "v");
    four(k, "k");
    four(v, "v");
    if (v.scalar_type() != k.scalar_type() || v.sizes() != k.sizes())
      fail("v: expected k's type and shape, got " + got(v));
    svsa_cache_tokens p{};
    p.dtype = dtype_of(k, "k");
    p.N = int32_of(k.size(2), "tokens");
    for (int e = 0; e < 3; ++e) {
      p.k_stride[e] = k.stride(e);
      p.v_stride[e] = v.stride(e);
    }
    return make(2, p);
  });
}

// cache_append(cache, k, v, n_new, len_out, params, stream)
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() {
    count(n, 7);
    Struct<svsa_cache> c(a[0], false, "c");
    Struct<svsa_cache_tokens> p(a[5], false, "p");
    const int dev = device_of(a[0]);
    const at::ScalarType type = type_of(p->dtype);
    void* k = view(tensor(a[1], "k"), type, {c->B, c->heads, p->N, c->d}, p->k_stride, dev, "k");
    void* v = view(tensor(a[2], "v"), type, {c->B, c->heads, p->N, c->d}, p->v_stride, dev, "v");
    void* n_new = dense(tensor(a[3], "n_new", true), at::kInt, {c->B}, dev, "n_new");
    void* len_out = dense(tensor(a[4], "len_out", true), at::kInt, {c->B}, dev, "len_out");
    Launch l(dev, a[6]);
    return PyLong_FromLong(svsa_cache_append(&*c, k, v, (int32_t*)n_new, (int32_t*)len_out, &*p, l.stream()));
  });
}

// cache_query(q, causal, cap, first, last)
PyObject* cache_query(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() {
    count(n, 5);
    const at::Tensor& q = *tensor(a[0], "q");
    four(q, "q");
    svsa_cache_query p{};
    p.dtype = dtype_of(q, "q");
    p.heads_q = int32_of(q.size(1), "heads");
    p.Tq = int32_of(q.size(2), "Tq");
    p.causal = truth(a[1]);
    p.cap = int32_of(integer(a[2]), "cap");
    p.first = int32_of(integer(a[3]), "first");
    p.last = int32_of(integer(a[4]), "last");
    return make(3, p);
  });
}

// cache_select(cache, q, idx, cnt, params, stream)
PyObject* cache_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() {
    count(n, 6);
    Struct<svsa_cache> c(a[0], false, "c");
    Struct<svsa_cache_query> p(a[4], false, "p");
    const int dev = device_of(a[0]);
    void* q = dense(tensor(a[1], "q"), type_of(p->dtype), {c->B, p->heads_q, p->Tq, c->d}, dev, "q");
    void* idx = dense(tensor(a[2], "idx"), at::kInt, {c->B, p->Tq, c->heads, p->cap}, dev, "idx");
    void* cnt = dense(tensor(a[3], "cnt"), at::kInt, {c->B, p->Tq, c->heads}, dev, "cnt");
    Launch l(dev, a[5]);
    return PyLong_FromLong(svsa_cache_select(&*c, q, (int32_t*)idx, (int32_t*)cnt, &*p, l.stream()));
  });
}

// cache_attn(cache, q, idx, cnt, o, lse, params, ws, ws_bytes, stream)
PyObject* cache_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() {
    count(n, 10);
    Struct<svsa_cache> c(a[0], false, "c");
    Struct<svsa_cache_query> p(a[6], false, "p");
    const int dev = device_of(a[0]);
    const at::ScalarType type = type_of(p->dtype);
    void* q = dense(tensor(a[1], "q"), type, {c->B, p->heads_q, p->Tq, c->d}, dev, "q");
    void* idx = dense(tensor(a[2], "idx", true), at::kInt, {c->B, p->Tq, c->heads, p->cap}, dev, "idx");
    void* cnt = dense(tensor(a[3], "cnt", true), at::kInt, {c->B, p->Tq, c->heads}, dev, "cnt");
    void* o = dense(tensor(a[4], "o"), type, {c->B, p->heads_q, p->Tq, c->d}, dev, "o");
    void* lse = dense(tensor(a[5], "lse", true), at::kFloat, {c->B, p->heads_q, p->Tq}, dev, "lse");
    const int64_t bytes = integer(a[8]);
    void* ws = workspace(tensor(a[7], "ws", true), bytes, dev);
    Launch l(dev, a[9]);
    return PyLong_FromLong(svsa_cache_attn(&*c, q, (int32_t*)idx, (int32_t*)cnt, o, (float*)lse, &*p, ws,
                                           (size_t)bytes, l.stream()));
  });
}

// cache_attn_workspace_bytes(cache, params)
PyObject* cache_attn_workspace_bytes(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() {
    count(n, 2);
    Struct<svsa_cache> c(a[0], false, "c");
    Struct<svsa_cache_query> p(a[1], false, "p");
    return PyLong_FromSize_t(svsa_cache_attn_workspace_bytes(&*c, &*p));
  });
}

// qk_norm_rope_bwd_workspace_bytes(params)
PyObject* rope_workspace(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() {
    count(n, 1);
    Struct<svsa_norm_rope> p(a[0], false, "p");
    return PyLong_FromSize_t(svsa_qk_norm_rope_bwd_workspace_bytes(&*p));
  });
}

// init(NormRopeParams, Cache, CacheTokens, CacheQuery): the package's ctypes structures
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() {
    count(n, 4);
    for (int i = 0; i < 4; ++i) {
      Py_INCREF(a[i]);
      Py_XSETREF(g_types[i], a[i]);
    }
    Py_RETURN_NONE;
  });
}

#define SVSA_METHOD(name, fn) {name, (PyCFunction)(void (*)(void))fn, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    SVSA_METHOD("init", init),
    SVSA_METHOD("norm_rope_params", norm_rope_params),
    SVSA_METHOD("qk_norm_rope", qk_norm_rope),
    SVSA_METHOD("qk_norm_rope_bwd_workspace_bytes", rope_workspace),
    SVSA_METHOD("qk_norm_rope_bwd", qk_norm_rope_bwd),
    SVSA_METHOD("block_cache", block_cache),
    SVSA_METHOD("cache_tokens", cache_tokens),
    SVSA_METHOD("cache_append", cache_append),
    SVSA_METHOD("cache_query", cache_query),
    SVSA_METHOD("cache_select", cache_select),
    SVSA_METHOD("cache_attn_workspace_bytes", cache_attn_workspace_bytes),
    SVSA_METHOD("cache_attn", cache_attn),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_svsa_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__svsa_binding(void) {
  g_device = PyUnicode_InternFromString("device");
  return g_device ? PyModule_Create(&module) : nullptr;
}
