// Python calls of the attention group: the checks of tensors and the hand-over of
// their pointers to the C ABI, as api.py documents them, in C++.
//
// These calls launch kernels of 3 to 10 us. Checking and passing some 30 arguments
// from Python takes 6 us a call, the launch itself 3.5; here the former takes under
// 1 (host time: one token's head norm 9.9 -> 4.2 us, the 4 calls of a step, which
// make their outputs, 41 -> 21).
#include <Python.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <exception>
#include <initializer_list>
#include <string>

#include "btq.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

struct Raised {};   // a Python exception is set

[[noreturn]] void raise(PyObject* type, const std::string& text) {
  PyErr_SetString(type, text.c_str());
  throw Raised{};
}

std::string text_of(IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + ": expected a tensor");
  return THPVariable_Unpack(o);
}

constexpr ScalarType kValues[] = {ScalarType::Float, ScalarType::BFloat16, ScalarType::Short};

void need_type(const Tensor& t, const char* name, std::initializer_list<ScalarType> types) {
  for (ScalarType s : types)
    if (t.scalar_type() == s) return;
  std::string want;
  for (ScalarType s : types) want += std::string(want.empty() ? "" : ", ") + c10::toString(s);
  raise(PyExc_TypeError, std::string(name) + ": dtype " + c10::toString(t.scalar_type()) +
                             ", expected one of " + want);
}
void need_value(const Tensor& t, const char* name) { need_type(t, name, {kValues[0], kValues[1], kValues[2]}); }

void need_shape(const Tensor& t, const char* name, IntArrayRef shape) {
  if (t.sizes() != shape)
    raise(PyExc_ValueError, std::string(name) + ": shape " + text_of(t.sizes()) + ", expected " + text_of(shape));
}

int gpu_of(const Tensor& t) {
  if (!t.is_cuda()) raise(PyExc_ValueError, "libbtq runs on the GPU: pass device tensors");
  return t.get_device();
}
void need_device(const Tensor& t, const char* name, int device) {
  if (!t.is_cuda() || t.get_device() != device)
    raise(PyExc_ValueError, std::string(name) + ": on " + t.device().str() + ", expected cuda:" + std::to_string(device));
}

// Data of a contiguous tensor, checked.
void* data(PyObject* o, const char* name, std::initializer_list<ScalarType> types, IntArrayRef shape, int device) {
  const Tensor& t = tensor(o, name);
  need_type(t, name, types);
  need_shape(t, name, shape);
  if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + ": must be contiguous");
  need_device(t, name, device);
  return t.data_ptr();
}

int value_type(const Tensor& t) { return t.scalar_type() == ScalarType::Float ? BTQ_T_F32 : BTQ_T_BF16; }

// Heads [T,heads,D] or [P,T,heads,D] whose last dimension is contiguous.
struct Rows {
  bool sharded;
  int64_t P, T, H, D, shard, pitch, head;
  void* p;
  int type;
};
Rows rows_of(const Tensor& t, const char* name) {
  const auto s = t.sizes(), st = t.strides();
  const size_t n = s.size();
  if (n != 3 && n != 4)
    raise(PyExc_ValueError, std::string(name) + ": shape " + text_of(s) + ", expected [T,heads,D] or [P,T,heads,D]");
  if (st[n - 1] != 1 && s[n - 1] > 1)
    raise(PyExc_ValueError, std::string(name) + ": the last dimension must be contiguous");
  return {n == 4, n == 4 ? s[0] : 1, s[n - 3], s[n - 2], s[n - 1], n == 4 ? st[0] : 0, st[n - 3], st[n - 2],
          t.data_ptr(), value_type(t)};
}
Rows like_rows(PyObject* o, const char* name, IntArrayRef shape, int device) {
  const Tensor& t = tensor(o, name);
  need_value(t, name);
  need_shape(t, name, shape);
  need_device(t, name, device);
  return rows_of(t, name);
}

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    raise(PyIndex_Check(o) ? PyExc_OverflowError : PyExc_TypeError,
          std::string(name) + ": expected an integer of 64 bits");
  }
  return v;
}
float number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    raise(PyExc_TypeError, std::string(name) + ": expected a number");
  }
  return (float)v;
}

int option(PyObject* o, const char* what, std::initializer_list<const char*> names) {
  int i = 0;
  if (PyUnicode_Check(o))
    for (const char* n : names) {
      if (PyUnicode_CompareWithASCIIString(o, n) == 0) return i;
      ++i;
    }
  std::string all;
  for (const char* n : names) all += std::string(all.empty() ? "" : ", ") + n;
  raise(PyExc_ValueError, std::string(what) + " must be among " + all);
}

struct Rope {
  const float *cos, *sin;
  int64_t rows, dim;
  int style;
};
Rope rope_of(PyObject* cos, PyObject* sin, PyObject* style, int device) {
  Rope r = {nullptr, nullptr, 0, 0, option(style, "rope", {"half", "pairs"})};
  if (cos == Py_None && sin == Py_None) return r;
  if (cos == Py_None || sin == Py_None || tensor(cos, "cos").dim() != 2)
    raise(PyExc_ValueError, "cos and sin: both or neither, [rows, rope_dim/2]");
  const Tensor& t = tensor(cos, "cos");
  r.cos = (const float*)data(cos, "cos", {ScalarType::Float}, t.sizes(), device);
  r.sin = (const float*)data(sin, "sin", {ScalarType::Float}, t.sizes(), device);
  r.rows = t.size(0);
  r.dim = 2 * t.size(1);
  return r;
}

struct Weight {
  const float* p;
  int64_t shard, head;
};
Weight weight_of(PyObject* o, const char* name, const Rows& x, int64_t heads, int device) {
  if (o == Py_None) return {nullptr, 0, 0};
  if (tensor(o, name).dim() == 1) return {(const float*)data(o, name, {ScalarType::Float}, {x.D}, device), 0, 0};
  void* p = x.sharded ? data(o, name, {ScalarType::Float}, {x.P, heads, x.D}, device)
                      : data(o, name, {ScalarType::Float}, {heads, x.D}, device);
  return {(const float*)p, heads * x.D, x.D};
}

// A batch of sequences and its cache, as every call of the group names them.
struct Batch {
  const int32_t *starts, *lengths, *table;
  int64_t B, max_pages;
  uint8_t* cache;
  int64_t pages, page_size, Hk, D;
};
Batch batch_of(PyObject* starts, PyObject* lengths, PyObject* table, PyObject* cache, bool sharded, int64_t P,
               int device) {
  const Tensor& c = tensor(cache, "cache");
  const auto s = c.sizes();
  if (s.size() != (sharded ? 5u : 4u))
    raise(PyExc_ValueError, "cache: shape " + text_of(s) + ", expected [" + (sharded ? "P," : "") +
                                "pages,Hk,page_size/32,block bytes]");
  if (sharded && s[0] != P)
    raise(PyExc_ValueError, "cache: " + std::to_string(s[0]) + " shards, the heads have " + std::to_string(P));
  const size_t n = s.size();
  Batch b;
  b.B = tensor(lengths, "lengths").dim() == 1 ? tensor(lengths, "lengths").size(0) : -1;
  b.max_pages = tensor(table, "page_table").dim() == 2 ? tensor(table, "page_table").size(1) : -1;
  b.starts = (const int32_t*)data(starts, "seq_starts", {ScalarType::Int}, {b.B + 1}, device);
  b.lengths = (const int32_t*)data(lengths, "lengths", {ScalarType::Int}, {b.B}, device);
  b.table = (const int32_t*)data(table, "page_table", {ScalarType::Int}, {b.B, b.max_pages}, device);
  b.cache = (uint8_t*)data(cache, "cache", {ScalarType::Byte}, s, device);
  b.pages = s[n - 4];
  b.Hk = s[n - 3];
  b.page_size = 32 * s[n - 2];
  b.D = s[n - 1] >= 256 && btq_kv_block_bytes((s[n - 1] - 256) / 32) == s[n - 1] ? (s[n - 1] - 256) / 32 : -1;
  if (b.D < 0) raise(PyExc_ValueError, "cache: no head has blocks of " + std::to_string(s[n - 1]) + " bytes");
  return b;
}

PyObject* g_current_stream = nullptr;   // torch._C._cuda_getCurrentRawStream

void* stream_of(PyObject* o, int device) {
  if (o != Py_None) return (void*)(intptr_t)integer(o, "stream");
  PyObject* index = PyLong_FromLong(device);
  PyObject* s = index ? PyObject_CallOneArg(g_current_stream, index) : nullptr;
  Py_XDECREF(index);
  if (!s) throw Raised{};
  void* p = PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  if (!p && PyErr_Occurred()) throw Raised{};
  return p;
}

void check(int status, const char* what) {
  if (status != BTQ_OK)
    raise(PyExc_RuntimeError,
          std::string(what) + ": " + btq_status_str(status) + " (status " + std::to_string(status) + ")");
}

ScalarType type_or(PyObject* o, ScalarType otherwise) {
  if (o == Py_None) return otherwise;
  if (!THPDtype_Check(o)) raise(PyExc_TypeError, "dtype: expected a torch.dtype");
  return ((THPDtype*)o)->scalar_type;
}
at::TensorOptions on(int device, ScalarType type) {
  return at::TensorOptions().dtype(type).device(c10::Device(c10::kCUDA, (c10::DeviceIndex)device));
}

// No C++ exception leaves a call.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (const Raised&) {
  } catch (...) {
    // torch's own, as its calls from Python raise them (torch.OutOfMemoryError, say)
    if (!PyErr_Occurred()) torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}
PyObject* same(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// (x, q_heads, norm, q_weight, k_weight, eps, positions, cos, sin, rope, out, out_dtype, stream)
PyObject* head_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    const Tensor& x = tensor(a[0], "x");
    const int device = gpu_of(x);
    need_value(x, "x");
    const Rows r = rows_of(x, "x");
    const int64_t q_heads = integer(a[1], "q_heads");
    const int norm = option(a[2], "norm", {"none", "rms", "layer"});
    if (q_heads < 0 || q_heads > r.H)
      raise(PyExc_ValueError, "q_heads: " + std::to_string(q_heads) + " of " + std::to_string(r.H) + " heads");
    const Weight q = weight_of(a[3], "q_weight", r, q_heads, device);
    const Weight k = weight_of(a[4], "k_weight", r, r.H - q_heads, device);
    const float eps = number(a[5], "eps");
    const Rope rope = rope_of(a[7], a[8], a[9], device);
    const int32_t* positions = nullptr;
    if (rope.cos) {
      if (a[6] == Py_None) raise(PyExc_ValueError, "positions: needed with cos and sin");
      positions = (const int32_t*)data(a[6], "positions", {ScalarType::Int}, {r.T}, device);
    }
    const c10::DeviceGuard guard(x.device());
    Tensor made;
    Rows y;
    if (a[10] == Py_None) {
      made = at::empty(x.sizes(), on(device, type_or(a[11], x.scalar_type())));
      need_value(made, "out");
      y = rows_of(made, "out");
    } else {
      y = like_rows(a[10], "out", x.sizes(), device);
    }
    check(btq_head_norm_rope(r.p, r.type, r.shard, r.pitch, r.head, r.P, r.T, q_heads, r.H - q_heads, r.D, norm, q.p,
                             q.shard, q.head, k.p, k.shard, k.head, eps, positions, rope.cos, rope.sin, rope.rows,
                             rope.dim, rope.style, y.p, y.type, y.shard, y.pitch, y.head, stream_of(a[12], device)),
          "btq_head_norm_rope");
    return a[10] == Py_None ? THPVariable_Wrap(made) : same(a[10]);
  });
}

// (k, v, seq_starts, lengths, page_table, cache, cos, sin, rope, stream)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const Tensor& kt = tensor(a[0], "k");
    const int device = gpu_of(kt);
    need_value(kt, "k");
    const Rows k = rows_of(kt, "k");
    const Tensor& vt = tensor(a[1], "v");
    need_type(vt, "v", {kt.scalar_type()});
    const Rows v = like_rows(a[1], "v", kt.sizes(), device);
    const Batch b = batch_of(a[2], a[3], a[4], a[5], k.sharded, k.P, device);
    if (k.H != b.Hk || k.D != b.D)
      raise(PyExc_ValueError, "k: " + std::to_string(k.H) + " heads of " + std::to_string(k.D) + ", the cache has " +
                                  std::to_string(b.Hk) + " of " + std::to_string(b.D));
    const Rope rope = rope_of(a[6], a[7], a[8], device);
    const c10::DeviceGuard guard(kt.device());
    check(btq_kv_append(k.p, v.p, k.type, k.shard, k.pitch, k.head, v.shard, v.pitch, v.head, k.P, k.T, k.H, k.D,
                        b.starts, b.lengths, b.B, b.table, b.max_pages, rope.cos, rope.sin, rope.rows, rope.dim,
                        rope.style, b.cache, b.pages, b.page_size, stream_of(a[9], device)),
          "btq_kv_append");
    Py_RETURN_NONE;
  });
}

// (seq_starts, lengths, page_table, cache, tokens, k, v, dtype, stream)
PyObject* kv_gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const Tensor& c = tensor(a[3], "cache");
    const int device = gpu_of(c);
    const bool sharded = c.dim() == 5;
    const int64_t P = sharded ? c.size(0) : 1;
    const Batch b = batch_of(a[0], a[1], a[2], a[3], sharded, P, device);
    const c10::DeviceGuard guard(c.device());
    Tensor made_k, made_v;
    PyObject *ko = a[5], *vo = a[6];
    Rows k = {}, v = {};
    int64_t T = 0;
    if (ko == Py_None && vo == Py_None) {
      if (a[4] == Py_None) raise(PyExc_ValueError, "tokens: needed without k and v");
      T = integer(a[4], "tokens");
      if (T < 0) raise(PyExc_ValueError, "tokens: must not be negative");
      const int64_t shape[4] = {P, T, b.Hk, b.D};
      const IntArrayRef s(shape + (sharded ? 0 : 1), sharded ? 4 : 3);
      made_k = at::zeros(s, on(device, type_or(a[7], ScalarType::BFloat16)));
      made_v = at::zeros(s, made_k.options());
      need_value(made_k, "dtype");
      k = rows_of(made_k, "k");
      v = rows_of(made_v, "v");
    } else {
      const Tensor& x = tensor(ko != Py_None ? ko : vo, ko != Py_None ? "k" : "v");
      T = x.dim() >= 3 ? x.size(-3) : -1;
      const int64_t shape[4] = {P, T, b.Hk, b.D};
      const IntArrayRef s(shape + (sharded ? 0 : 1), sharded ? 4 : 3);
      if (ko != Py_None) k = like_rows(ko, "k", s, device);
      if (vo != Py_None) {
        v = like_rows(vo, "v", s, device);
        if (ko != Py_None) need_type(tensor(vo, "v"), "v", {x.scalar_type()});
      }
    }
    check(btq_kv_gather(b.starts, b.lengths, b.B, b.table, b.max_pages, b.cache, b.pages, b.page_size, P, T, b.Hk, b.D,
                        k.p, v.p, k.p ? k.type : v.type, k.shard, k.pitch, k.head, v.shard, v.pitch, v.head,
                        stream_of(a[8], device)),
          "btq_kv_gather");
    PyObject* first = made_k.defined() ? THPVariable_Wrap(made_k) : same(ko);
    PyObject* second = made_v.defined() ? THPVariable_Wrap(made_v) : same(vo);
    PyObject* pair = PyTuple_Pack(2, first, second);
    Py_XDECREF(first);
    Py_XDECREF(second);
    return pair;
  });
}

// (q, seq_starts, lengths, page_table, cache, scale, causal, window, max_length, out, out_dtype, lse,
//  workspace, stream)
PyObject* kv_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const Tensor& qt = tensor(a[0], "q");
    const int device = gpu_of(qt);
    need_type(qt, "q", {ScalarType::BFloat16, ScalarType::Short});
    const Rows q = rows_of(qt, "q");
    const Batch b = batch_of(a[1], a[2], a[3], a[4], q.sharded, q.P, device);
    if (q.D != b.D || b.Hk < 1 || q.H % b.Hk)
      raise(PyExc_ValueError, "q: " + std::to_string(q.H) + " heads of " + std::to_string(q.D) + ", the cache has " +
                                  std::to_string(b.Hk) + " of " + std::to_string(b.D));
    const float scale = a[5] == Py_None ? (float)(1.0 / std::sqrt((double)q.D)) : number(a[5], "scale");
    const int causal = PyObject_IsTrue(a[6]);
    if (causal < 0) throw Raised{};
    const int64_t window = integer(a[7], "window"), max_length = integer(a[8], "max_length");
    const c10::DeviceGuard guard(qt.device());
    const int64_t shape[3] = {q.P, q.T, q.H * q.D}, sums[3] = {q.P, q.T, q.H};
    const size_t skip = q.sharded ? 0 : 1;
    const IntArrayRef s(shape + skip, 3 - skip);
    Tensor made, scratch;
    void* out;
    int out_type;
    if (a[9] == Py_None) {
      made = at::zeros(s, on(device, type_or(a[10], qt.scalar_type())));
      need_value(made, "out");
      out = made.data_ptr();
      out_type = value_type(made);
    } else {
      out = data(a[9], "out", {kValues[0], kValues[1], kValues[2]}, s, device);
      out_type = value_type(tensor(a[9], "out"));
    }
    float* lse = a[11] == Py_None ? nullptr
                                  : (float*)data(a[11], "lse", {ScalarType::Float}, IntArrayRef(sums + skip, 3 - skip), device);
    const size_t need = btq_kv_attention_workspace_bytes(q.P, q.T, q.H, b.Hk, q.D, b.B, b.max_pages, b.page_size, max_length);
    void* ws = nullptr;
    size_t bytes = 0;
    if (a[12] != Py_None) {
      const Tensor& w = tensor(a[12], "workspace");
      if (!w.is_cuda() || w.get_device() != device || !w.is_contiguous())
        raise(PyExc_ValueError, "workspace: must be contiguous and on cuda:" + std::to_string(device));
      ws = w.data_ptr();
      bytes = w.nbytes();
    } else if (need) {
      scratch = at::empty({(int64_t)need}, on(device, ScalarType::Byte));
      ws = scratch.data_ptr();
      bytes = need;
    }
    check(btq_kv_attention(q.p, q.shard, q.pitch, q.head, q.P, q.T, q.H, b.Hk, q.D, b.starts, b.lengths, b.B, b.table,
                           b.max_pages, b.cache, b.pages, b.page_size, scale, causal, window, max_length, out, out_type,
                           lse, ws, bytes, stream_of(a[13], device)),
          "btq_kv_attention");
    return made.defined() ? THPVariable_Wrap(made) : same(a[9]);
  });
}

PyMethodDef g_methods[] = {{"head_norm_rope", (PyCFunction)(void*)head_norm_rope, METH_FASTCALL, nullptr},
                           {"kv_append", (PyCFunction)(void*)kv_append, METH_FASTCALL, nullptr},
                           {"kv_gather", (PyCFunction)(void*)kv_gather, METH_FASTCALL, nullptr},
                           {"kv_attention", (PyCFunction)(void*)kv_attention, METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* c = PyImport_ImportModule("torch._C");
  if (!c) return nullptr;
  g_current_stream = PyObject_GetAttrString(c, "_cuda_getCurrentRawStream");
  Py_DECREF(c);
  // (a torch without GPU support has no streams; then no call gets as far)
  if (!g_current_stream) {
    PyErr_Clear();
    g_current_stream = same(Py_None);
  }
  return PyModule_Create(&g_module);
}
