// Argument marshalling for the windowed and the cached calls: torch tensors in,
// the C ABI of fa_b200.h out.  It does what the Python binding would do -- check
// types, shapes, devices and strides, allocate outputs, fetch the current stream
// -- in C++, because these calls are made per layer and token and the Python form
// cost more than the kernels of a small one (one new token, 12 heads, context
// 1000: 18 us of host time against 11 us on the GPU; 7 us here).  No step of an operator is
// computed here, and the library is the one that _abi.py has loaded: bind()
// receives the addresses of its entry points.
//
// Every function raises TypeError or ValueError for arguments that do not fit,
// and returns the library's status (first, where outputs follow) otherwise.
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/Exceptions.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstring>
#include <string>

#include "fa_b200.h"

namespace {

struct Library {
  decltype(&fa_window_fwd) window_fwd;
  decltype(&fa_window_bwd) window_bwd;
  decltype(&fa_window_bwd_workspace_bytes) window_bwd_workspace_bytes;
  decltype(&fa_cached_fwd) cached_fwd;
  decltype(&fa_cached_workspace_bytes) cached_workspace_bytes;
  decltype(&fa_cache_append) cache_append;
  decltype(&fa_cache_compact) cache_compact;
} lib{};

struct Refused {};  // a Python error is set

using at::Tensor;

const Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", name);
    throw Refused();
  }
  return THPVariable_Unpack(o);
}

std::string listed(at::IntArrayRef v) {
  std::string s = "(";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + ")";
}

[[noreturn]] void refuse(const char* name, const Tensor& t, at::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
  const std::string s = std::string(name) + " must be a " + c10::toString(type) + " tensor of shape " + listed(shape) +
                        " on " + dev.str() + ", contiguous (views: along the last axis), got " +
                        c10::toString(t.scalar_type()) + " " + listed(t.sizes()) + " on " + t.device().str() +
                        (t.layout() == at::kStrided ? ", strides " + listed(t.strides()) : ", not strided");
  PyErr_SetString(PyExc_ValueError, s.c_str());
  throw Refused();
}

// contiguous tensor of that shape, type and device -> its data
template <typename T = void>
T* vec(const char* name, PyObject* o, at::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
  const Tensor& t = tensor(name, o);
  if (t.scalar_type() != type || t.device() != dev || t.sizes() != shape || !t.is_contiguous() || t.layout() != at::kStrided)
    refuse(name, t, shape, type, dev);
  return static_cast<T*>(t.data_ptr());
}

fa_view view_of(const Tensor& t) { return {t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)}; }

// bf16 tensor of that shape and device whose last axis is contiguous -> its view
fa_view view(const char* name, PyObject* o, at::IntArrayRef shape, c10::Device dev) {
  const Tensor& t = tensor(name, o);
  if (t.scalar_type() != at::kBFloat16 || t.device() != dev || t.sizes() != shape || t.layout() != at::kStrided ||
      t.stride(3) != 1)
    refuse(name, t, shape, at::kBFloat16, dev);
  return view_of(t);
}

// the tensor whose shape and device the others follow
const Tensor& leading(const char* name, PyObject* o) {
  const Tensor& t = tensor(name, o);
  if (t.dim() != 4 || !t.is_cuda()) {
    PyErr_Format(PyExc_ValueError, "%s must be a four-dimensional CUDA bfloat16 tensor", name);
    throw Refused();
  }
  return t;
}

int whole(PyObject* o, const char* name, long long least) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  if (v < least || v > 2147483647ll) {
    PyErr_Format(PyExc_ValueError, "%s must be in [%lld, 2**31 - 1], got %lld", name, least, v);
    throw Refused();
  }
  return static_cast<int>(v);
}

// sizes that are passed as C ints
int extent(int64_t v) {
  if (v > 2147483647ll) {
    PyErr_Format(PyExc_ValueError, "an axis of %lld entries is beyond the library's domain", static_cast<long long>(v));
    throw Refused();
  }
  return static_cast<int>(v);
}

struct Softmax {
  int window, sinks, mode;
  float beta;
};
Softmax softmax(PyObject* const* a) {  // window, sinks, softmax_mode, beta
  Softmax s{whole(a[0], "window", 1), whole(a[1], "sinks", 0), 0, 0.f};
  const long mode = PyLong_AsLong(a[2]);
  if (mode == -1 && PyErr_Occurred()) throw Refused();
  s.mode = mode >= -1 && mode <= 1000 ? static_cast<int>(mode) : -1;
  const double beta = PyFloat_AsDouble(a[3]);
  if (beta == -1.0 && PyErr_Occurred()) throw Refused();
  s.beta = static_cast<float>(beta);
  return s;
}

PyObject* wrap(Tensor t) { return THPVariable_Wrap(std::move(t)); }

// (status, tensors...)
template <typename... T>
PyObject* result(int status, T... t) {
  PyObject* items[] = {PyLong_FromLong(status), wrap(t)...};
  constexpr Py_ssize_t n = 1 + sizeof...(T);
  PyObject* r = PyTuple_New(n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (r && items[i])
      PyTuple_SET_ITEM(r, i, items[i]);
    else {
      Py_XDECREF(items[i]);
      Py_CLEAR(r);
    }
  }
  return r;
}

// The library call without the interpreter lock, on the tensors' device and its
// current stream.
template <typename F>
int run(c10::Device dev, F call) {
  const c10::cuda::CUDAGuard guard(dev);
  void* stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = call(stream);
  Py_END_ALLOW_THREADS
  return status;
}

Tensor bytes(size_t n, c10::Device dev) {
  return at::empty({static_cast<int64_t>(n)}, at::TensorOptions().device(dev).dtype(at::kByte));
}
Tensor floats(at::IntArrayRef shape, c10::Device dev) {
  return at::empty(shape, at::TensorOptions().device(dev).dtype(at::kFloat));
}

// ------------------------------------------------------------------ windowed
struct WindowShapes {
  int64_t q[4], kv[4], rows[3];
  int B, H, Hkv, N, d;
  c10::Device dev;
  WindowShapes(const Tensor& t, PyObject* k)
      : B(extent(t.size(0))), H(extent(t.size(1))), Hkv(-1), N(extent(t.size(2))), d(extent(t.size(3))), dev(t.device()) {
    const Tensor& kt = tensor("k", k);
    if (kt.dim() == 4) Hkv = extent(kt.size(1));
    for (int i = 0; i < 4; ++i) q[i] = t.size(i);
    kv[0] = B, kv[1] = Hkv, kv[2] = N, kv[3] = d;
    rows[0] = B, rows[1] = H, rows[2] = N;
  }
};

int window_fwd_call(const WindowShapes& s, PyObject* const* qkv, const fa_view& o, float* lse, const fa_row_stats* st,
                    const Softmax& x) {
  const fa_view q = view("q", qkv[0], s.q, s.dev), k = view("k", qkv[1], s.kv, s.dev), v = view("v", qkv[2], s.kv, s.dev);
  return run(s.dev, [&](void* stream) {
    return lib.window_fwd(&q, &k, &v, &o, lse, st, s.B, s.H, s.Hkv, s.N, s.d, x.window, x.sinks, x.mode, x.beta, stream);
  });
}

// q, k, v, o, lse, rm, rs, m, pbar_max (each of the four may be None), window, sinks, softmax_mode, beta
PyObject* window_fwd(PyObject* const* a) {
  const Softmax x = softmax(a + 9);
  const WindowShapes s(leading("q", a[0]), a[1]);
  const fa_view o = view("o", a[3], s.q, s.dev);
  float* lse = vec<float>("lse", a[4], s.rows, at::kFloat, s.dev);
  fa_row_stats st{};
  if (a[5] != Py_None) st.rm = vec<float>("stats.rm", a[5], s.rows, at::kFloat, s.dev);
  if (a[6] != Py_None) st.rs = vec<int32_t>("stats.rs", a[6], s.rows, at::kInt, s.dev);
  if (a[7] != Py_None) st.m = vec<float>("stats.m", a[7], s.rows, at::kFloat, s.dev);
  if (a[8] != Py_None) st.pbar_max = vec<float>("stats.pbar_max", a[8], s.rows, at::kFloat, s.dev);
  return PyLong_FromLong(window_fwd_call(s, a, o, lse, &st, x));
}

// q, k, v, window, sinks, softmax_mode, beta, with_stats -> status, o, lse[, rm, rs, m, pbar_max]
PyObject* window_forward(PyObject* const* a) {
  const Softmax x = softmax(a + 3);
  const Tensor& q = leading("q", a[0]);
  const WindowShapes s(q, a[1]);
  view("q", a[0], s.q, s.dev);
  Tensor o = at::empty_like(q), lse = floats(s.rows, s.dev);
  if (a[7] != Py_True) return result(window_fwd_call(s, a, view_of(o), lse.data_ptr<float>(), nullptr, x), o, lse);
  // m, which the backward needs, on its own; the others in one allocation
  const int64_t all[4] = {3, s.rows[0], s.rows[1], s.rows[2]};
  Tensor rows = floats(all, s.dev), m = floats(s.rows, s.dev);
  Tensor rm = rows.select(0, 0), rs = rows.select(0, 1).view(at::kInt), pbar = rows.select(0, 2);
  const fa_row_stats st{rm.data_ptr<float>(), rs.data_ptr<int32_t>(), m.data_ptr<float>(), pbar.data_ptr<float>()};
  return result(window_fwd_call(s, a, view_of(o), lse.data_ptr<float>(), &st, x), o, lse, rm, rs, m, pbar);
}

int window_bwd_call(const WindowShapes& s, PyObject* const* a, const fa_view& dq, const fa_view& dk, const fa_view& dv,
                    void* ws, size_t ws_bytes, const Softmax& x) {
  const fa_view q = view("q", a[0], s.q, s.dev), k = view("k", a[1], s.kv, s.dev), v = view("v", a[2], s.kv, s.dev);
  const fa_view o = view("o", a[3], s.q, s.dev), dO = view("dO", a[4], s.q, s.dev);
  const float* lse = vec<float>("lse", a[5], s.rows, at::kFloat, s.dev);
  const float* row_m = a[6] == Py_None ? nullptr : vec<float>("row_m", a[6], s.rows, at::kFloat, s.dev);
  return run(s.dev, [&](void* stream) {
    return lib.window_bwd(&q, &k, &v, &o, &dO, lse, row_m, &dq, &dk, &dv, ws, ws_bytes, s.B, s.H, s.Hkv, s.N, s.d,
                          x.window, x.sinks, x.mode, x.beta, stream);
  });
}

// a uint8 tensor of one axis -> pointer and size
void* workspace(PyObject* o, c10::Device dev, size_t* size) {
  const Tensor& t = tensor("workspace", o);
  const int64_t n = t.numel();
  *size = static_cast<size_t>(n);
  return vec("workspace", o, at::IntArrayRef(n), at::kByte, dev);
}

// q, k, v, o, dO, lse, row_m, dq, dk, dv, workspace, window, sinks, softmax_mode, beta
PyObject* window_bwd(PyObject* const* a) {
  const Softmax x = softmax(a + 11);
  const WindowShapes s(leading("q", a[0]), a[1]);
  size_t size = 0;
  void* ws = workspace(a[10], s.dev, &size);
  return PyLong_FromLong(window_bwd_call(s, a, view("dq", a[7], s.q, s.dev), view("dk", a[8], s.kv, s.dev),
                                         view("dv", a[9], s.kv, s.dev), ws, size, x));
}

// q, k, v, o, dO, lse, row_m, workspace or None, window, sinks, softmax_mode, beta -> status, dq, dk, dv, workspace
PyObject* window_backward(PyObject* const* a) {
  const Softmax x = softmax(a + 8);
  const Tensor& q = leading("q", a[0]);
  const WindowShapes s(q, a[1]);
  view("q", a[0], s.q, s.dev);
  view("k", a[1], s.kv, s.dev);
  view("v", a[2], s.kv, s.dev);
  Tensor ws;
  if (a[7] == Py_None) {
    const c10::cuda::CUDAGuard guard(s.dev);
    ws = bytes(lib.window_bwd_workspace_bytes(s.B, s.H, s.Hkv, s.N, s.d, x.window, x.sinks), s.dev);
  } else {
    ws = tensor("workspace", a[7]);
  }
  size_t size = static_cast<size_t>(ws.numel());
  void* at_ws = a[7] == Py_None ? ws.data_ptr() : workspace(a[7], s.dev, &size);
  Tensor dq = at::empty_like(q), dk = at::empty_like(tensor("k", a[1])), dv = at::empty_like(tensor("v", a[2]));
  return result(window_bwd_call(s, a, view_of(dq), view_of(dk), view_of(dv), at_ws, size, x), dq, dk, dv, ws);
}

// -------------------------------------------------------------------- cache
struct Pool {
  void *k, *v;
  const int32_t *table, *ctx;
  int B, Hkv, d, pages, page, width;
};
// k_pages, v_pages, page_table, ctx_len
Pool pool(PyObject* const* a, c10::Device dev) {
  const Tensor &k = tensor("k_pages", a[0]), &table = tensor("page_table", a[2]);
  if (k.dim() != 4 || table.dim() != 2) {
    PyErr_SetString(PyExc_ValueError,
                    "k_pages must be a bfloat16 tensor [num_pages, Hkv, page_size, d], page_table an int32 tensor "
                    "[B, table_width]");
    throw Refused();
  }
  Pool p{};
  p.k = vec("k_pages", a[0], k.sizes(), at::kBFloat16, dev);
  p.v = vec("v_pages", a[1], k.sizes(), at::kBFloat16, dev);
  p.table = vec<int32_t>("page_table", a[2], table.sizes(), at::kInt, dev);
  p.ctx = vec<int32_t>("ctx_len", a[3], at::IntArrayRef(table.size(0)), at::kInt, dev);
  p.pages = extent(k.size(0)), p.Hkv = extent(k.size(1)), p.page = extent(k.size(2)), p.d = extent(k.size(3));
  p.B = extent(table.size(0)), p.width = extent(table.size(1));
  return p;
}

[[noreturn]] void unlike(const char* what, const Tensor& t, const Pool& p) {
  const std::string s = std::string(what) + " is " + listed(t.sizes()) + ", the cache has " + std::to_string(p.B) +
                        " sequences, " + std::to_string(p.Hkv) + " heads and rows of " + std::to_string(p.d);
  PyErr_SetString(PyExc_ValueError, s.c_str());
  throw Refused();
}

// q, k_pages, v_pages, page_table, ctx_len, tree or None
int cached_call(const Tensor& q, PyObject* const* a, const Pool& p, const fa_view& o, float* lse, void* ws, size_t size,
                const Softmax& x) {
  const c10::Device dev = q.device();
  const int B = p.B, H = extent(q.size(1)), T = extent(q.size(2));
  const fa_view vq = view("q", a[0], q.sizes(), dev);
  const int64_t words[2] = {B, T};
  const int64_t* tree = a[5] == Py_None ? nullptr : vec<int64_t>("tree", a[5], words, at::kLong, dev);
  return run(dev, [&](void* stream) {
    return lib.cached_fwd(&vq, p.k, p.v, p.table, p.ctx, reinterpret_cast<const uint64_t*>(tree), &o, lse, ws, size, B, H,
                          p.Hkv, T, p.d, p.pages, p.page, p.width, x.window, x.sinks, x.mode, x.beta, stream);
  });
}

// q, k_pages, v_pages, page_table, ctx_len, tree or None, o, lse, workspace, window, sinks, softmax_mode, beta
PyObject* cached_fwd(PyObject* const* a) {
  const Softmax x = softmax(a + 9);
  const Tensor& q = leading("q", a[0]);
  const Pool p = pool(a + 1, q.device());
  if (q.size(0) != p.B || q.size(3) != p.d) unlike("q", q, p);
  const int64_t rows[3] = {q.size(0), q.size(1), q.size(2)};
  size_t size = 0;
  void* ws = workspace(a[8], q.device(), &size);
  return PyLong_FromLong(cached_call(q, a, p, view("o", a[6], q.sizes(), q.device()),
                                     vec<float>("lse", a[7], rows, at::kFloat, q.device()), ws, size, x));
}

// q, k_pages, v_pages, page_table, ctx_len, tree or None, workspace or None, window, sinks, softmax_mode, beta
// -> status, o, lse
PyObject* cached(PyObject* const* a) {
  const Softmax x = softmax(a + 7);
  const Tensor& q = leading("q", a[0]);
  const Pool p = pool(a + 1, q.device());
  if (q.size(0) != p.B || q.size(3) != p.d) unlike("q", q, p);
  view("q", a[0], q.sizes(), q.device());
  Tensor own;
  size_t size = 0;
  void* ws;
  if (a[6] == Py_None) {
    size = lib.cached_workspace_bytes(p.B, extent(q.size(1)), p.Hkv, extent(q.size(2)), p.d);
    own = bytes(size, q.device());
    ws = own.data_ptr();
  } else {
    ws = workspace(a[6], q.device(), &size);
  }
  const int64_t rows[3] = {q.size(0), q.size(1), q.size(2)};
  Tensor o = at::empty_like(q), lse = floats(rows, q.device());
  return result(cached_call(q, a, p, view_of(o), lse.data_ptr<float>(), ws, size, x), o, lse);
}

// k, v, k_pages, v_pages, page_table, ctx_len, count or None
PyObject* append(PyObject* const* a) {
  const Tensor& k = leading("k", a[0]);
  const c10::Device dev = k.device();
  const Pool p = pool(a + 2, dev);
  if (k.size(0) != p.B || k.size(1) != p.Hkv || k.size(3) != p.d) unlike("k", k, p);
  const fa_view vk = view("k", a[0], k.sizes(), dev), vv = view("v", a[1], k.sizes(), dev);
  const int32_t* count = a[6] == Py_None ? nullptr : vec<int32_t>("count", a[6], at::IntArrayRef(k.size(0)), at::kInt, dev);
  const int T = extent(k.size(2));
  return PyLong_FromLong(run(dev, [&](void* stream) {
    return lib.cache_append(&vk, &vv, p.k, p.v, p.table, p.ctx, count, p.B, p.Hkv, T, p.d, p.pages, p.page, p.width,
                            stream);
  }));
}

// k_pages, v_pages, page_table, ctx_len, src, count
PyObject* compact(PyObject* const* a) {
  const Tensor& k = leading("k_pages", a[0]);
  const c10::Device dev = k.device();
  const Pool p = pool(a, dev);
  const Tensor& st = tensor("src", a[4]);
  const int M = st.dim() == 2 ? extent(st.size(1)) : -1;
  const int64_t moves[2] = {p.B, M};
  const int32_t* src = vec<int32_t>("src", a[4], moves, at::kInt, dev);
  const int32_t* count = vec<int32_t>("count", a[5], at::IntArrayRef(moves, 1), at::kInt, dev);
  return PyLong_FromLong(run(dev, [&](void* stream) {
    return lib.cache_compact(p.k, p.v, p.table, p.ctx, src, count, p.B, p.Hkv, M, p.d, p.pages, p.page, p.width, stream);
  }));
}

// the library's addresses, in the order of Library
PyObject* bind(PyObject* const* a) {
  void* at[7];
  for (int i = 0; i < 7; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i]);
    if (!at[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null entry point");
      throw Refused();
    }
  }
  static_assert(sizeof(Library) == sizeof(at), "one address per entry point");
  std::memcpy(&lib, at, sizeof(lib));
  Py_RETURN_NONE;
}

// No C++ exception leaves a call: torch's become Python's, the rest RuntimeError.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N, bool BOUND = true>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
    return nullptr;
  }
  if (BOUND && !lib.window_fwd) {
    PyErr_SetString(PyExc_RuntimeError, "the library is not loaded");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N, bool BOUND = true>
constexpr PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N, BOUND>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<bind, 7, false>("bind"),
    method<window_fwd, 13>("window_fwd"),
    method<window_forward, 8>("window_forward"),
    method<window_bwd, 15>("window_bwd"),
    method<window_backward, 12>("window_backward"),
    method<cached_fwd, 13>("cached_fwd"),
    method<cached, 11>("cached"),
    method<append, 7>("append"),
    method<compact, 6>("compact"),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "tensor marshalling for libfa_b200.so", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
