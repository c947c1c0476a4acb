// paged_binding.cpp -- the paged cache's calls from Python: reads the layer,
// the batch and the tensors, checks them and calls the C ABI.
//
// A generation step's kernels take a few microseconds, and checking a dozen
// tensors from Python takes longer than that; here it takes a microsecond
// (a call of attn_paged_move 7.8 -> 3.4 us of host time). No computation and
// no state: the C functions' addresses come from the package, which has loaded
// the library.
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstdarg>
#include <string>

#include "../../include/cswattn.h"

namespace {

using AppendFn = decltype(&attn_paged_append);
using AttendFn = decltype(&attn_paged);
using WeighFn = decltype(&attn_paged_weigh);
using SelectFn = decltype(&attn_paged_select);
using MoveFn = decltype(&attn_paged_move);
using ErrorFn = decltype(&cswattn_last_error);

struct {
  AppendFn append;
  AttendFn attend;
  WeighFn weigh;
  SelectFn select;
  MoveFn move;
  ErrorFn last_error;
  PyObject* error;  // CswattnError(status, message)
} g{};

// Thrown behind a set Python exception; nothing passes the module's functions.
struct Raised {};

[[noreturn]] __attribute__((format(printf, 2, 3))) void raise(PyObject* type, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(type, fmt, ap);
  va_end(ap);
  throw Raised{};
}

// An owned reference.
struct Ref {
  PyObject* p;
  explicit Ref(PyObject* p_) : p(p_) {
    if (!p) throw Raised{};
  }
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
  Ref(Ref&& o) noexcept : p(o.p) { o.p = nullptr; }
  ~Ref() { Py_XDECREF(p); }
};

// Interned attribute names, made once.
struct Names {
  PyObject *B, *T, *n_head, *n_kv_head, *head_dim, *window, *has_ve, *dtype, *rope_base, *eps, *softmax_scale;
  PyObject *page_table, *cache_len, *new_start, *n_tokens, *max_new;
  PyObject *k, *v, *weight, *position, *n_pages, *page_size, *address, *cuda_stream;
} n;

Ref attr(PyObject* o, PyObject* name) { return Ref(PyObject_GetAttr(o, name)); }

int to_int(PyObject* o, const char* what) {
  const long x = PyLong_AsLong(o);
  if (x == -1 && PyErr_Occurred()) throw Raised{};
  if (x < INT_MIN || x > INT_MAX) raise(PyExc_ValueError, "%s does not fit 32 bits", what);
  return static_cast<int>(x);
}
int int_attr(PyObject* o, PyObject* name) { return to_int(attr(o, name).p, PyUnicode_AsUTF8(name)); }
float float_attr(PyObject* o, PyObject* name) {
  const double x = PyFloat_AsDouble(attr(o, name).p);
  if (x == -1.0 && PyErr_Occurred()) throw Raised{};
  return static_cast<float>(x);
}

cswattn_layer read_layer(PyObject* spec) {
  cswattn_layer l;
  l.B = int_attr(spec, n.B);
  l.T = int_attr(spec, n.T);
  l.n_head = int_attr(spec, n.n_head);
  l.n_kv_head = int_attr(spec, n.n_kv_head);
  l.head_dim = int_attr(spec, n.head_dim);
  l.window = int_attr(spec, n.window);
  l.rope_base = float_attr(spec, n.rope_base);
  l.eps = float_attr(spec, n.eps);
  l.softmax_scale = float_attr(spec, n.softmax_scale);
  const int ve = PyObject_IsTrue(attr(spec, n.has_ve).p);
  if (ve < 0) throw Raised{};
  l.has_ve = ve;
  const Ref dt = attr(spec, n.dtype);
  l.dtype = PyUnicode_Check(dt.p) && PyUnicode_CompareWithASCIIString(dt.p, "bf16") == 0 ? CSWATTN_BF16 : CSWATTN_F32;
  return l;
}

constexpr auto kBf16 = at::kBFloat16;
constexpr auto kF32 = at::kFloat;
constexpr auto kI32 = at::kInt;

std::string dims(at::IntArrayRef a) {
  std::string s = "(";
  for (size_t i = 0; i < a.size(); ++i) s += (i ? ", " : "") + std::to_string(a[i]);
  return s + ")";
}

// The address of a contiguous CUDA tensor of this type and shape on the
// device (which the first tensor of a call sets when it is -1).
void* want(const char* name, PyObject* o, at::ScalarType type, at::IntArrayRef shape, int& device) {
  if (o == Py_None) raise(PyExc_ValueError, "%s is needed", name);
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a tensor, got %s", name, Py_TYPE(o)->tp_name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) raise(PyExc_ValueError, "%s must be a CUDA tensor", name);
  const int on = t.get_device();
  if (device < 0) device = on;
  if (on != device)
    raise(PyExc_ValueError, "%s lies on cuda:%d, other tensors of the call on cuda:%d", name, on, device);
  if (t.scalar_type() != type) {
    raise(PyExc_ValueError, "%s must be %s, got %s", name, c10::toString(type), c10::toString(t.scalar_type()));
  }
  if (t.sizes() != shape) {
    const std::string want_ = dims(shape), got = dims(t.sizes());
    raise(PyExc_ValueError, "%s must have shape %s, got %s", name, want_.c_str(), got.c_str());
  }
  if (!t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
  return t.data_ptr();
}
void* want_or_null(const char* name, PyObject* o, at::ScalarType type, at::IntArrayRef shape, int& device) {
  return o == Py_None ? nullptr : want(name, o, type, shape, device);
}

// Scratch: any type and shape. Its bytes are *bytes unless the caller gave a number.
void* want_scratch(PyObject* o, PyObject* given, int& device, size_t* bytes) {
  *bytes = 0;
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "workspace must be a tensor, got %s", Py_TYPE(o)->tp_name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous())
    raise(PyExc_ValueError, "workspace must be a contiguous CUDA tensor on the call's device");
  *bytes = t.nbytes();
  if (given != Py_None) {
    const size_t x = PyLong_AsSize_t(given);
    if (x == static_cast<size_t>(-1) && PyErr_Occurred()) throw Raised{};
    if (x < *bytes) *bytes = x;  // never more than there is
  }
  return t.data_ptr();
}

struct Call {
  cswattn_layer layer;
  cswattn_paged paged;
  int device = -1;
  int64_t B, H, Hk, D, pages, page, N;

  Call(PyObject* spec, PyObject* batch, PyObject* cache) : layer(read_layer(spec)) {
    B = layer.B;
    H = layer.n_head;
    Hk = layer.n_kv_head;
    D = layer.head_dim;
    paged.page_size = int_attr(cache, n.page_size);
    paged.n_pages = int_attr(cache, n.n_pages);
    paged.n_tokens = int_attr(batch, n.n_tokens);
    paged.max_new = int_attr(batch, n.max_new);
    pages = paged.n_pages;
    page = paged.page_size;
    N = paged.n_tokens;
    const Ref table = attr(batch, n.page_table), len = attr(batch, n.cache_len), start = attr(batch, n.new_start);
    if (!THPVariable_Check(table.p) || THPVariable_Unpack(table.p).dim() != 2)
      raise(PyExc_ValueError, "page_table must be a tensor (sequences, pages)");
    const int64_t rows = THPVariable_Unpack(table.p).size(0), cols = THPVariable_Unpack(table.p).size(1);
    if (rows != B)
      raise(PyExc_ValueError, "the batch has %lld sequences, the layer %lld", static_cast<long long>(rows),
            static_cast<long long>(B));
    paged.pages_per_seq = cols > INT_MAX ? INT_MAX : static_cast<int>(cols);
    paged.page_table = static_cast<int*>(want("page_table", table.p, kI32, {B, cols}, device));
    paged.cache_len = static_cast<int*>(want("cache_len", len.p, kI32, {B}, device));
    paged.new_start = static_cast<int*>(want_or_null("new_start", start.p, kI32, {B + 1}, device));
  }
  // A pool of the cache (null if it has none and `needed` is false).
  void* pool(PyObject* cache, PyObject* name, bool rows, bool needed) {
    const Ref t = attr(cache, name);
    const char* s = PyUnicode_AsUTF8(name);
    if (t.p == Py_None && needed) raise(PyExc_ValueError, "the cache has no %s", s);
    const at::ScalarType type = rows ? kBf16 : (name == n.weight ? kF32 : kI32);
    return rows ? want_or_null(s, t.p, type, {pages, page, Hk, D}, device)
                : want_or_null(s, t.p, type, {pages, Hk, page}, device);
  }
};

// Calls fn(stream) with the tensors' device current and raises its error.
template <class Fn>
PyObject* run(int device, PyObject* stream, const Fn& fn) {
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(device));
  void* st;
  if (stream == Py_None) {
    st = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  } else if (PyLong_Check(stream)) {
    st = PyLong_AsVoidPtr(stream);
  } else {
    const Ref handle = attr(stream, n.cuda_stream);
    st = PyLong_AsVoidPtr(handle.p);
  }
  if (PyErr_Occurred()) throw Raised{};
  const cswattn_status status = fn(st);
  if (status == CSWATTN_OK) Py_RETURN_NONE;
  const Ref e(PyObject_CallFunction(g.error, "is", static_cast<int>(status), g.last_error()));
  PyErr_SetObject(g.error, e.p);
  throw Raised{};
}

// A module function: a fixed number of positional arguments, no exception out.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t count) {
  if (count != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments are wanted, got %zd", N, count);
    return nullptr;
  }
  if (!g.error) {
    PyErr_SetString(PyExc_RuntimeError, "bind() first");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// (n_kv_head, head_dim, k, v, weight, position) -> (n_pages, page_size)
PyObject* check_cache(PyObject* const* a) {
  const int64_t Hk = to_int(a[0], "n_kv_head"), D = to_int(a[1], "head_dim");
  const bool rows = a[2] != Py_None || a[3] != Py_None;
  PyObject* lead = a[2] != Py_None ? a[2] : (a[3] != Py_None ? a[3] : (a[4] != Py_None ? a[4] : a[5]));
  if (lead == Py_None) raise(PyExc_ValueError, "PagedCache needs n_pages and page_size, or the pools");
  if (!THPVariable_Check(lead) || THPVariable_Unpack(lead).dim() != (rows ? 4 : 3))
    raise(PyExc_ValueError, "a pool must be a tensor of %d dimensions", rows ? 4 : 3);
  const int64_t pages = THPVariable_Unpack(lead).size(0), page = THPVariable_Unpack(lead).size(rows ? 1 : 2);
  int device = -1;
  want_or_null("k", a[2], kBf16, {pages, page, Hk, D}, device);
  want_or_null("v", a[3], kBf16, {pages, page, Hk, D}, device);
  want_or_null("weight", a[4], kF32, {pages, Hk, page}, device);
  want_or_null("position", a[5], kI32, {pages, Hk, page}, device);
  return Py_BuildValue("LL", static_cast<long long>(pages), static_cast<long long>(page));
}

// (page_table, cache_len, new_start)
PyObject* check_batch(PyObject* const* a) {
  if (!THPVariable_Check(a[0]) || THPVariable_Unpack(a[0]).dim() != 2)
    raise(PyExc_ValueError, "page_table must be a tensor (sequences, pages)");
  const int64_t B = THPVariable_Unpack(a[0]).size(0), cols = THPVariable_Unpack(a[0]).size(1);
  int device = -1;
  want("page_table", a[0], kI32, {B, cols}, device);
  want("cache_len", a[1], kI32, {B}, device);
  want_or_null("new_start", a[2], kI32, {B + 1}, device);
  Py_RETURN_NONE;
}

// (spec, batch, cache, q, k, v, ve, gate, q_out, positions, rope, stream)
PyObject* append(PyObject* const* a) {
  Call c(a[0], a[1], a[2]);
  const int64_t N = c.N, H = c.H, Hk = c.Hk, D = c.D;
  const void* q = want("q", a[3], kBf16, {N, H, D}, c.device);
  const void* k = want("k", a[4], kBf16, {N, Hk, D}, c.device);
  const void* v = want("v", a[5], kBf16, {N, Hk, D}, c.device);
  const bool has_ve = c.layer.has_ve != 0;
  const void* ve = has_ve ? want("ve", a[6], kBf16, {N, Hk, D}, c.device) : nullptr;
  const void* gate = has_ve ? want("gate", a[7], kBf16, {N, Hk}, c.device) : nullptr;
  void* q_out = want("q_out", a[8], kBf16, {N, H, D}, c.device);
  const int* pos = static_cast<int*>(want_or_null("positions", a[9], kI32, {N}, c.device));
  const cswattn_rope* rope = nullptr;
  if (a[10] != Py_None) {
    rope = static_cast<const cswattn_rope*>(PyLong_AsVoidPtr(attr(a[10], n.address).p));
    if (PyErr_Occurred()) throw Raised{};
  }
  void* kp = c.pool(a[2], n.k, true, true);
  void* vp = c.pool(a[2], n.v, true, true);
  float* w = static_cast<float*>(c.pool(a[2], n.weight, false, false));
  int* p = static_cast<int*>(c.pool(a[2], n.position, false, false));
  return run(c.device, a[11], [&](void* st) {
    return g.append(&c.layer, &c.paged, rope, q, k, v, ve, gate, pos, q_out, kp, vp, w, p, st);
  });
}

// (spec, batch, cache, q_out, O, lse, workspace, workspace_bytes, stream)
PyObject* attend(PyObject* const* a) {
  Call c(a[0], a[1], a[2]);
  const void* q = want("q_out", a[3], kBf16, {c.N, c.H, c.D}, c.device);
  void* O = want("O", a[4], kBf16, {c.N, c.H, c.D}, c.device);
  float* lse = static_cast<float*>(want("lse", a[5], kF32, {c.N, c.H}, c.device));
  size_t bytes;
  void* ws = want_scratch(a[6], a[7], c.device, &bytes);
  void* kp = c.pool(a[2], n.k, true, true);
  void* vp = c.pool(a[2], n.v, true, true);
  return run(c.device, a[8],
             [&](void* st) { return g.attend(&c.layer, &c.paged, q, kp, vp, O, lse, ws, bytes, st); });
}

// (spec, batch, cache, q_out, lse, workspace, stream)
PyObject* weigh(PyObject* const* a) {
  Call c(a[0], a[1], a[2]);
  const void* q = want("q_out", a[3], kBf16, {c.N, c.H, c.D}, c.device);
  const float* lse = static_cast<float*>(want("lse", a[4], kF32, {c.N, c.H}, c.device));
  size_t bytes;
  void* ws = want_scratch(a[5], Py_None, c.device, &bytes);
  void* kp = c.pool(a[2], n.k, true, true);
  float* w = static_cast<float*>(c.pool(a[2], n.weight, false, true));
  return run(c.device, a[6],
             [&](void* st) { return g.weigh(&c.layer, &c.paged, q, kp, lse, w, ws, bytes, st); });
}

// (spec, batch, cache, next_pos, n_keep, n_recent, n_moves, src, dst, new_len, stream)
PyObject* select(PyObject* const* a) {
  Call c(a[0], a[1], a[2]);
  const int keep = to_int(a[4], "n_keep"), recent = to_int(a[5], "n_recent");
  const int* next = static_cast<int*>(want("next_pos", a[3], kI32, {c.B}, c.device));
  int* moves = static_cast<int*>(want("n_moves", a[6], kI32, {c.B, c.Hk}, c.device));
  int* src = static_cast<int*>(want("src", a[7], kI32, {c.B, c.Hk, keep}, c.device));
  int* dst = static_cast<int*>(want("dst", a[8], kI32, {c.B, c.Hk, keep}, c.device));
  int* len = static_cast<int*>(want("new_len", a[9], kI32, {c.B}, c.device));
  const float* w = static_cast<float*>(c.pool(a[2], n.weight, false, true));
  const int* p = static_cast<int*>(c.pool(a[2], n.position, false, true));
  return run(c.device, a[10], [&](void* st) {
    return g.select(&c.layer, &c.paged, w, p, next, keep, recent, moves, src, dst, len, st);
  });
}

// (spec, batch, cache, n_moves, src, dst, stream)
PyObject* move(PyObject* const* a) {
  Call c(a[0], a[1], a[2]);
  if (!THPVariable_Check(a[4]) || THPVariable_Unpack(a[4]).dim() != 3)
    raise(PyExc_ValueError, "src must be a tensor (sequences, n_kv_head, n_keep)");
  const int64_t keep = THPVariable_Unpack(a[4]).size(2);
  const int* moves = static_cast<int*>(want("n_moves", a[3], kI32, {c.B, c.Hk}, c.device));
  const int* src = static_cast<int*>(want("src", a[4], kI32, {c.B, c.Hk, keep}, c.device));
  const int* dst = static_cast<int*>(want("dst", a[5], kI32, {c.B, c.Hk, keep}, c.device));
  void* kp = c.pool(a[2], n.k, true, true);
  void* vp = c.pool(a[2], n.v, true, true);
  float* w = static_cast<float*>(c.pool(a[2], n.weight, false, true));
  int* p = static_cast<int*>(c.pool(a[2], n.position, false, true));
  return run(c.device, a[6], [&](void* st) {
    return g.move(&c.layer, &c.paged, moves, src, dst, keep > INT_MAX ? INT_MAX : static_cast<int>(keep), kp, vp, w, p,
                  st);
  });
}

// bind(CswattnError, addresses of append, attend, weigh, select, move, last_error)
PyObject* bind(PyObject*, PyObject* args) {
  PyObject *error, *f[6];
  if (!PyArg_ParseTuple(args, "OOOOOOO", &error, &f[0], &f[1], &f[2], &f[3], &f[4], &f[5])) return nullptr;
  void* p[6];
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(f[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is 0");
      return nullptr;
    }
  }
  g.append = reinterpret_cast<AppendFn>(p[0]);
  g.attend = reinterpret_cast<AttendFn>(p[1]);
  g.weigh = reinterpret_cast<WeighFn>(p[2]);
  g.select = reinterpret_cast<SelectFn>(p[3]);
  g.move = reinterpret_cast<MoveFn>(p[4]);
  g.last_error = reinterpret_cast<ErrorFn>(p[5]);
  Py_INCREF(error);
  Py_XSETREF(g.error, error);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr},
                         method<check_cache, 6>("check_cache"),
                         method<check_batch, 3>("check_batch"),
                         method<append, 12>("append"),
                         method<attend, 9>("attend"),
                         method<weigh, 7>("weigh"),
                         method<select, 11>("select"),
                         method<move, 7>("move"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_binding() {
  struct {
    PyObject** to;
    const char* name;
  } names[] = {{&n.B, "B"}, {&n.T, "T"}, {&n.n_head, "n_head"}, {&n.n_kv_head, "n_kv_head"}, {&n.head_dim, "head_dim"},
               {&n.window, "window"}, {&n.has_ve, "has_ve"}, {&n.dtype, "dtype"}, {&n.rope_base, "rope_base"},
               {&n.eps, "eps"}, {&n.softmax_scale, "softmax_scale"}, {&n.page_table, "page_table"},
               {&n.cache_len, "cache_len"}, {&n.new_start, "new_start"}, {&n.n_tokens, "n_tokens"},
               {&n.max_new, "max_new"}, {&n.k, "k"}, {&n.v, "v"}, {&n.weight, "weight"}, {&n.position, "position"},
               {&n.n_pages, "n_pages"}, {&n.page_size, "page_size"}, {&n.address, "address"},
               {&n.cuda_stream, "cuda_stream"}};
  for (const auto& x : names) {
    *x.to = PyUnicode_InternFromString(x.name);
    if (!*x.to) return nullptr;
  }
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", BUILT_FOR) < 0) Py_CLEAR(m);
  return m;
}
