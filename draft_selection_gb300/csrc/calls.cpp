// The Python side of the cache and tree calls: types and shapes of the tensors, which
// the C side cannot see, are checked here, and their addresses, strides and sizes handed
// to libdfl2.so.  A call is a few microseconds of GPU time, and marshalling it in Python
// took the host as long again: a turn of one sequence, five calls, 40.8 us a pass, 25.2
// so; one token's attention 11.9 and 9.2.  Arguments are positional; the functions of
// the package name them.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <exception>
#include <initializer_list>

#include "dfl2.h"

namespace {

struct Raised {};  // the Python exception is set

#define REFUSE(type, ...)               \
  do {                                  \
    PyErr_Format(type, __VA_ARGS__);    \
    throw Raised();                     \
  } while (0)

using Sizes = std::initializer_list<int64_t>;

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o))
    REFUSE(PyExc_TypeError, "%s must be a tensor, not %s", name, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o, const char* name, int dims) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != dims)
    REFUSE(PyExc_ValueError, "%s must have %d dimensions, not %lld", name, dims,
           (long long)t.dim());
  return t;
}
bool has_shape(const at::Tensor& t, Sizes shape) {
  return t.sizes() == at::IntArrayRef(shape);
}
// An int32 device array's address; None: NULL.
int32_t* i32(PyObject* o, const char* name, Sizes shape) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kInt) REFUSE(PyExc_TypeError, "%s must be int32", name);
  if (!has_shape(t, shape) || !t.is_contiguous()) {
    PyObject* want = PyTuple_New(0);
    for (int64_t n : shape) {
      PyObject* one = Py_BuildValue("(L)", (long long)n);
      PyObject* more = one && want ? PySequence_Concat(want, one) : nullptr;
      Py_XDECREF(one);
      Py_XDECREF(want);
      want = more;
    }
    if (want) PyErr_Format(PyExc_ValueError, "%s must be contiguous %R", name, want);
    Py_XDECREF(want);
    throw Raised();
  }
  return static_cast<int32_t*>(t.data_ptr());
}
int whole(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  if (v < INT_MIN || v > INT_MAX) REFUSE(PyExc_OverflowError, "%s is out of range", name);
  return static_cast<int>(v);
}
// Sizes are ints in the C calls.
int size(const at::Tensor& t, int i, const char* name) {
  if (t.size(i) > INT_MAX) REFUSE(PyExc_OverflowError, "%s is too large", name);
  return static_cast<int>(t.size(i));
}
const dfl2_cache* cache_of(PyObject* o) {
  static PyObject* name = PyUnicode_InternFromString("_address");
  PyObject* a = PyObject_GetAttr(o, name);
  if (!a) throw Raised();
  void* p = PyLong_AsVoidPtr(a);
  Py_DECREF(a);
  if (!p) REFUSE(PyExc_TypeError, "no cache");
  return static_cast<const dfl2_cache*>(p);
}
at::ScalarType type_of(const dfl2_cache* c) {
  return c->dtype == DFL2_F32 ? at::kFloat : c->dtype == DFL2_BF16 ? at::kBFloat16 : at::kHalf;
}
// None: torch's current stream; else an address or a torch stream.
dfl2_stream stream_of(PyObject* o) {
  if (o == Py_None)
    return reinterpret_cast<dfl2_stream>(c10::cuda::getCurrentCUDAStream().stream());
  PyObject* a = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
  if (!a) throw Raised();
  void* p = PyLong_AsVoidPtr(a);
  Py_DECREF(a);
  if (!p && PyErr_Occurred()) throw Raised();
  return reinterpret_cast<dfl2_stream>(p);
}
// Equal but for dimensions of one entry, whose strides torch leaves open.
bool same_strides(const at::Tensor& a, const at::Tensor& b) {
  for (int64_t i = 0; i < a.dim(); ++i)
    if (a.size(i) != 1 && a.stride(i) != b.stride(i)) return false;
  return true;
}

// The call itself, without the interpreter's lock; the status.
template <typename F>
PyObject* run(F f) {
  dfl2_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = f();
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

PyObject* cache_reserve(PyObject* const* a) {  // cache, length, count, served, rows, stream
  const dfl2_cache* c = cache_of(a[0]);
  const at::Tensor& len = tensor(a[1], "length", 1);
  const int B = size(len, 0, "length");
  if (a[2] == Py_None) REFUSE(PyExc_TypeError, "count must be a number or int32 [B]");
  const bool same = PyLong_Check(a[2]);  // one count for all
  const int T = same ? whole(a[2], "count") : 1 << 30;
  const int32_t* n = same ? nullptr : i32(a[2], "count", {B});
  int32_t* served = i32(a[3], "served", {B});
  const int32_t* rows = i32(a[4], "rows", {B});
  const int32_t* length = i32(a[1], "length", {B});
  const dfl2_stream s = stream_of(a[5]);
  return run([&] { return dfl2_cache_reserve(c, B, T, rows, length, n, served, s); });
}

PyObject* cache_write(PyObject* const* a) {  // cache, k, v, length, count, rows, layer, stream
  const dfl2_cache* c = cache_of(a[0]);
  const at::Tensor &k = tensor(a[1], "k_new"), &v = tensor(a[2], "v_new");
  const int d = static_cast<int>(k.dim()), o = d - 4;  // o: where the sequences' dimension is
  if ((d != 4 && d != 5) || k.scalar_type() != type_of(c) || v.scalar_type() != type_of(c) ||
      v.sizes() != k.sizes() || k.size(d - 2) != c->kv_heads || k.size(d - 1) != c->head_dim)
    REFUSE(PyExc_ValueError,
           "k_new and v_new must be [n_layers, B, T, kv_heads, head_dim] of the cache's type");
  if (!same_strides(k, v) || k.stride(d - 1) != 1)
    REFUSE(PyExc_ValueError, "k_new and v_new must have the same strides, the last of them 1");
  const int N = o ? size(k, 0, "k_new") : 1, B = size(k, o, "k_new");
  int T = size(k, o + 1, "k_new");
  const int64_t st[4] = {o ? k.stride(0) : 0, k.stride(o), k.stride(o + 1), k.stride(o + 2)};
  const int32_t* n = nullptr;
  if (PyLong_Check(a[4]))
    T = std::min(T, whole(a[4], "count"));
  else
    n = i32(a[4], "count", {B});
  const int32_t *length = i32(a[3], "length", {B}), *rows = i32(a[5], "rows", {B});
  const int layer = whole(a[6], "layer");
  const void *kp = k.data_ptr(), *vp = v.data_ptr();
  const dfl2_stream s = stream_of(a[7]);
  return run([&] { return dfl2_cache_write(c, layer, N, kp, vp, st, B, T, rows, length, n, s); });
}

PyObject* cache_compact(PyObject* const* a) {
  // cache, length, count, path, n_path, new_length, rows, stream
  const dfl2_cache* c = cache_of(a[0]);
  const at::Tensor& p = tensor(a[3], "path", 2);
  const int B = size(p, 0, "path"), T = size(p, 1, "path");
  const int32_t* n = nullptr;
  if (!PyLong_Check(a[2])) {
    n = i32(a[2], "count", {B});
  } else if (whole(a[2], "count") != T) {
    REFUSE(PyExc_ValueError, "path has room for %d nodes, not %d", T, whole(a[2], "count"));
  }
  const int32_t *length = i32(a[1], "length", {B}), *path = i32(a[3], "path", {B, T}),
                *n_path = i32(a[4], "n_path", {B}), *rows = i32(a[6], "rows", {B});
  int32_t* new_length = i32(a[5], "new_length", {B});
  const dfl2_stream s = stream_of(a[7]);
  return run([&] {
    return dfl2_cache_compact(c, B, T, rows, length, n, path, n_path, new_length, s);
  });
}

PyObject* cache_fork(PyObject* const* a) {  // cache, src, dst, length, served, stream
  const dfl2_cache* c = cache_of(a[0]);
  const int n = size(tensor(a[1], "src", 1), 0, "src");
  const int32_t *src = i32(a[1], "src", {n}), *dst = i32(a[2], "dst", {n}),
                *length = i32(a[3], "length", {n});
  int32_t* served = i32(a[4], "served", {n});
  const dfl2_stream s = stream_of(a[5]);
  return run([&] { return dfl2_cache_fork(c, n, src, dst, length, served, s); });
}

PyObject* cache_free(PyObject* const* a) {  // cache, rows, stream
  const dfl2_cache* c = cache_of(a[0]);
  const int n = size(tensor(a[1], "rows", 1), 0, "rows");
  const int32_t* rows = i32(a[1], "rows", {n});
  const dfl2_stream s = stream_of(a[2]);
  return run([&] { return dfl2_cache_free(c, n, rows, s); });
}

PyObject* tree_mask(PyObject* const* a) {  // parents, mask, depth, count, stream
  const at::Tensor& p = tensor(a[0], "parents", 2);
  const int B = size(p, 0, "parents"), T = size(p, 1, "parents");
  const int32_t *parents = i32(a[0], "parents", {B, T}), *n = i32(a[3], "count", {B});
  int32_t *mask = i32(a[1], "mask", {B, T, (T + 31ll) / 32}), *depth = i32(a[2], "depth", {B, T});
  const dfl2_stream s = stream_of(a[4]);
  return run([&] {
    return dfl2_tree_mask(parents, B, T, n, reinterpret_cast<uint32_t*>(mask), depth, s);
  });
}

PyObject* tree_accept(PyObject* const* a) {
  // tokens, parents, target, path, n_path, next_token, count, stream
  const at::Tensor& t = tensor(a[0], "tokens", 2);
  const int B = size(t, 0, "tokens"), T = size(t, 1, "tokens");
  const int32_t *tokens = i32(a[0], "tokens", {B, T}), *parents = i32(a[1], "parents", {B, T}),
                *target = i32(a[2], "target", {B, T}), *n = i32(a[6], "count", {B});
  int32_t *path = i32(a[3], "path", {B, T}), *n_path = i32(a[4], "n_path", {B}),
          *next = i32(a[5], "next_token", {B});
  const dfl2_stream s = stream_of(a[7]);
  return run([&] {
    return dfl2_tree_accept(tokens, parents, target, B, T, n, path, n_path, next, s);
  });
}

// A float32 device array's address.
float* f32(PyObject* o, const char* name, Sizes shape) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kFloat) REFUSE(PyExc_TypeError, "%s must be float32", name);
  if (!has_shape(t, shape) || !t.is_contiguous())
    REFUSE(PyExc_ValueError, "%s must be contiguous, of the shape that the others give it", name);
  return static_cast<float*>(t.data_ptr());
}

PyObject* cache_evict(PyObject* const* a) {
  // cache, length, keep, sinks, recent, weight, kept, new_length, served, ws, rows, stream
  const dfl2_cache* c = cache_of(a[0]);
  const int B = size(tensor(a[1], "length", 1), 0, "length");
  const int keep = whole(a[2], "keep"), sinks = whole(a[3], "sinks"), recent = whole(a[4], "recent");
  const at::Tensor& ws = tensor(a[9], "ws");
  float* w = f32(a[5], "weight", {c->rows, int64_t(c->cols) * c->page_size});
  const int32_t *length = i32(a[1], "length", {B}), *rows = i32(a[10], "rows", {B});
  int32_t *kept = i32(a[6], "kept", {B, keep}), *new_length = i32(a[7], "new_length", {B}),
          *served = i32(a[8], "served", {B});
  void* wp = ws.data_ptr();
  const size_t bytes = ws.nbytes();
  const dfl2_stream s = stream_of(a[11]);
  return run([&] {
    return dfl2_cache_evict(c, B, rows, length, keep, sinks, recent, w, kept, new_length, served,
                            wp, bytes, s);
  });
}

PyObject* tree_verify(PyObject* const* a) {
  // p, tokens, parents, cand_idx, q, u, path, n_path, next_token, count, replace, stream
  const at::Tensor& p = tensor(a[0], "p", 3);
  const int B = size(p, 0, "p"), T = size(p, 1, "p"), V = size(p, 2, "p");
  const float* pp = f32(a[0], "p", {B, T, V});
  const int32_t *tokens = i32(a[1], "tokens", {B, T}), *parents = i32(a[2], "parents", {B, T}),
                *cand = i32(a[3], "cand_idx", {B, T, 16}), *n = i32(a[9], "count", {B});
  const float *q = f32(a[4], "q", {B, T, 16}), *u = f32(a[5], "u", {B, T});
  int32_t *path = i32(a[6], "path", {B, T}), *n_path = i32(a[7], "n_path", {B}),
          *next = i32(a[8], "next_token", {B});
  const int replace = PyObject_IsTrue(a[10]);
  if (replace < 0) throw Raised();
  const dfl2_stream s = stream_of(a[11]);
  return run([&] {
    return dfl2_tree_verify(pp, B, T, V, tokens, parents, n, cand, q, u, replace, path, n_path,
                            next, s);
  });
}

double scale_of(PyObject* o, const dfl2_cache* c) {
  if (o == Py_None) return std::pow(static_cast<double>(c->head_dim), -0.5);
  const double scale = PyFloat_AsDouble(o);
  if (scale == -1. && PyErr_Occurred()) throw Raised();
  return scale;
}

// q, cache, layer, length, mask, out, ws, rows, count, lse, scale, stream; win: then depth,
// sinks, window
PyObject* attn(PyObject* const* a, bool win) {
  const dfl2_cache* c = cache_of(a[1]);
  const at::Tensor &q = tensor(a[0], "q", 4), &out = tensor(a[5], "out", 4),
                   &ws = tensor(a[6], "ws");
  if (q.scalar_type() != type_of(c) || out.scalar_type() != type_of(c) || out.sizes() != q.sizes())
    REFUSE(PyExc_ValueError, "q and out must be [B, T, q_heads, head_dim] of the cache's type");
  if (q.size(3) != c->head_dim || q.stride(3) != 1 || out.stride(3) != 1)
    REFUSE(PyExc_ValueError, "q and out must have the cache's head_dim (%d, not %lld), stride 1",
           (int)c->head_dim, (long long)q.size(3));
  const int B = size(q, 0, "q"), T = size(q, 1, "q"), H = size(q, 2, "q");
  const int64_t qs[3] = {q.stride(0), q.stride(1), q.stride(2)},
                os[3] = {out.stride(0), out.stride(1), out.stride(2)};
  float* lse = nullptr;
  if (a[9] != Py_None) {
    const at::Tensor& t = tensor(a[9], "lse");
    if (t.scalar_type() != at::kFloat || !has_shape(t, {B, T, H}) || !t.is_contiguous())
      REFUSE(PyExc_ValueError, "lse must be contiguous float32 [B, T, q_heads]");
    lse = static_cast<float*>(t.data_ptr());
  }
  const double scale = scale_of(a[10], c);
  const int layer = whole(a[2], "layer");
  const int32_t *length = i32(a[3], "length", {B}),
                *mask = i32(a[4], "mask", {B, T, (T + 31ll) / 32}),
                *rows = i32(a[7], "rows", {B}), *n = i32(a[8], "count", {B});
  const void* qp = q.data_ptr();
  void *op = out.data_ptr(), *wp = ws.data_ptr();
  const size_t bytes = ws.nbytes();
  const int32_t* depth = win ? i32(a[12], "depth", {B, T}) : nullptr;
  const int sinks = win ? whole(a[13], "sinks") : 0, window = win ? whole(a[14], "window") : 0;
  const dfl2_stream s = stream_of(a[11]);
  return run([&] {
    const uint32_t* m = reinterpret_cast<const uint32_t*>(mask);
    if (win)
      return dfl2_window_attn(qp, qs, c, layer, B, T, H, rows, length, n, m, depth, sinks, window,
                              static_cast<float>(scale), op, os, lse, wp, bytes, s);
    return dfl2_tree_attn(qp, qs, c, layer, B, T, H, rows, length, n, m, static_cast<float>(scale), op,
                          os, lse, wp, bytes, s);
  });
}
PyObject* tree_attn(PyObject* const* a) { return attn(a, false); }
PyObject* window_attn(PyObject* const* a) { return attn(a, true); }

// Scratch of one call from torch's allocator, given back when the call has been issued: what
// the stream does next with the memory comes after it.
struct Scratch {
  void* p = nullptr;
  size_t bytes = 0;
  Scratch(size_t n, dfl2_stream s) : bytes(n) {
    if (n)
      p = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(n,
                                                                 reinterpret_cast<cudaStream_t>(s));
  }
  ~Scratch() {
    if (p) c10::cuda::CUDACachingAllocator::raw_delete(p);
  }
  Scratch(const Scratch&) = delete;
  Scratch& operator=(const Scratch&) = delete;
};

PyObject* cache_weigh(PyObject* const* a) {
  // q, lse, cache, layer, length, weight, ws (... where it is left out), path, n_path, first,
  // rows, scale, stream
  const dfl2_cache* c = cache_of(a[2]);
  const at::Tensor& q = tensor(a[0], "q", 4);
  const bool own = a[6] == Py_Ellipsis;
  const at::Tensor* ws = own ? nullptr : &tensor(a[6], "ws");
  if (q.scalar_type() != type_of(c))
    REFUSE(PyExc_ValueError, "q must be [B, T, q_heads, head_dim] of the cache's type");
  if (q.size(3) != c->head_dim || q.stride(3) != 1)
    REFUSE(PyExc_ValueError, "q must have the cache's head_dim (%d, not %lld), stride 1",
           (int)c->head_dim, (long long)q.size(3));
  const int B = size(q, 0, "q"), T = size(q, 1, "q"), H = size(q, 2, "q");
  const int64_t qs[3] = {q.stride(0), q.stride(1), q.stride(2)};
  const float* lse = f32(a[1], "lse", {B, T, H});
  float* weight = f32(a[5], "weight", {c->rows, int64_t(c->cols) * c->page_size});
  const double scale = scale_of(a[11], c);
  const int layer = whole(a[3], "layer"), first = PyObject_IsTrue(a[9]);
  if (first < 0) throw Raised();
  const int32_t *length = i32(a[4], "length", {B}), *path = i32(a[7], "path", {B, T}),
                *n_path = i32(a[8], "n_path", {B}), *rows = i32(a[10], "rows", {B});
  const void* qp = q.data_ptr();
  const dfl2_stream s = stream_of(a[12]);
  // (host memory is refused by the call)
  const Scratch scratch(own && q.is_cuda() ? dfl2_cache_weigh_workspace_size() : 0, s);
  void* wp = own ? scratch.p : ws->data_ptr();
  const size_t bytes = own ? scratch.bytes : ws->nbytes();
  return run([&] {
    return dfl2_cache_weigh(qp, qs, lse, c, layer, B, T, H, rows, length, path, n_path,
                            static_cast<float>(scale), first, weight, wp, bytes, s);
  });
}

// A function of N positional arguments; no C++ exception leaves it.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N) return PyErr_Format(PyExc_TypeError, "%d arguments, not %zd", N, n);
  try {
    return F(a);
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}
template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<cache_reserve, 6>("cache_reserve"),
                         method<cache_write, 8>("cache_write"),
                         method<cache_compact, 8>("cache_compact"),
                         method<cache_fork, 6>("cache_fork"),
                         method<cache_free, 3>("cache_free"),
                         method<tree_mask, 5>("tree_mask"),
                         method<tree_accept, 8>("tree_accept"),
                         method<cache_evict, 12>("cache_evict"),
                         method<tree_verify, 12>("tree_verify"),
                         method<tree_attn, 12>("tree_attn"),
                         method<window_attn, 15>("window_attn"),
                         method<cache_weigh, 13>("cache_weigh"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                      nullptr,               nullptr,  nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
