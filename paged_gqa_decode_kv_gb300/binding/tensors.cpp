// tensors.cpp -- the tensor side of the binding's calls on the block-scaled
// cache and on block selections: checks torch tensors against the types,
// shapes and device that a call takes and hands their addresses to libpgd.
//
// These calls run for two to five microseconds on the GPU at a decode step's
// sizes; checking and converting a dozen tensors in Python took three to five
// times as long.  Every function returns the library's status (an int), or with
// pack = True the arguments that it would have called with, as a tuple.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>
#include <string>

#include "pgd.h"

namespace {

constexpr int64_t kDim = 128;

struct Refused {};  // a Python exception is set

const char *dtype_name(at::ScalarType t) {
  switch (t) {
    case at::kByte: return "torch.uint8";
    case at::kChar: return "torch.int8";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kFloat: return "torch.float32";
    case at::kDouble: return "torch.float64";
    case at::kHalf: return "torch.float16";
    case at::kBFloat16: return "torch.bfloat16";
    default: return c10::toString(t);
  }
}

template <typename S>
std::string shape_text(const S &shape) {
  std::string s = "[";
  for (int64_t n : shape) s += (s.size() > 1 ? ", " : "") + std::to_string(n);
  return s + "]";
}

[[noreturn]] void refuse(PyObject *type, const std::string &what) {
  PyErr_SetString(type, what.c_str());
  throw Refused();
}

const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o))
    refuse(PyExc_TypeError, std::string(name) + " must be a tensor, got " + Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

// A tensor of `dims` dims (and, if given, of type `dtype`), for its sizes.
c10::IntArrayRef sizes(PyObject *o, int64_t dims, const char *name,
                       at::ScalarType dtype = at::ScalarType::Undefined) {
  const at::Tensor &t = tensor(o, name);
  if (dtype != at::ScalarType::Undefined && t.scalar_type() != dtype)
    refuse(PyExc_TypeError, std::string(name) + " must be " + dtype_name(dtype) + ", got " +
                                dtype_name(t.scalar_type()));
  if (t.dim() != dims)
    refuse(PyExc_ValueError, std::string(name) + " must be a tensor of " + std::to_string(dims) +
                                 " dims, got " + shape_text(t.sizes()));
  return t.sizes();
}

// The sizes as the library takes them.
int32_t int32(int64_t n, const char *what) {
  if (n < INT32_MIN || n > INT32_MAX)
    refuse(PyExc_ValueError, std::string(what) + " = " + std::to_string(n) + " does not fit int32");
  return (int32_t)n;
}
int64_t integer(PyObject *o, const char *what) {
  const long long n = PyLong_AsLongLong(o);
  if (n == -1 && PyErr_Occurred()) throw Refused();
  return int32(n, what);
}
float real(PyObject *o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Refused();
  return (float)x;
}

// Checks against one device (the first tensor's).
struct Args {
  int dev = -2;

  void *take(PyObject *o, at::ScalarType dtype, std::initializer_list<int64_t> shape,
             const char *name) {
    return take(o, dtype, c10::IntArrayRef(shape.begin(), shape.size()), name);
  }
  void *take(PyObject *o, at::ScalarType dtype, c10::IntArrayRef shape, const char *name) {
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != dtype)
      refuse(PyExc_TypeError, std::string(name) + " must be " + dtype_name(dtype) + ", got " +
                                  dtype_name(t.scalar_type()));
    if (t.sizes() != shape)
      refuse(PyExc_ValueError, std::string(name) + " must be " + shape_text(shape) + ", got " +
                                   shape_text(t.sizes()));
    return place(t, name);
  }
  void *take_opt(PyObject *o, at::ScalarType dtype, std::initializer_list<int64_t> shape,
                 const char *name) {
    return o == Py_None ? nullptr : take(o, dtype, shape, name);
  }
  // A contiguous tensor on the call's device: its address.
  void *place(const at::Tensor &t, const char *name) {
    if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
    if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be on a CUDA device");
    if (dev == -2) dev = t.get_device();
    if (t.get_device() != dev)
      refuse(PyExc_ValueError, std::string(name) + " is on cuda:" + std::to_string(t.get_device()) +
                                   ", the call on cuda:" + std::to_string(dev));
    return t.data_ptr();
  }
  // The given stream, or the current one; the library launches on the current
  // device, which must be the tensors'.
  void *stream(PyObject *o) const {
    const int cur = c10::cuda::current_device();
    if (cur != dev)
      refuse(PyExc_ValueError, "the tensors are on cuda:" + std::to_string(dev) +
                                   ", the current device is cuda:" + std::to_string(cur));
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    PyObject *s = PyObject_GetAttrString(o, "cuda_stream");
    if (!s) throw Refused();
    void *p = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    if (!p && PyErr_Occurred()) throw Refused();
    return p;
  }
};

PyObject *to_py(const void *p) {
  if (!p) Py_RETURN_NONE;
  return PyLong_FromVoidPtr(const_cast<void *>(p));
}
PyObject *to_py(int32_t n) { return PyLong_FromLong(n); }
PyObject *to_py(size_t n) { return PyLong_FromSize_t(n); }
PyObject *to_py(float x) { return PyFloat_FromDouble((double)x); }

// Calls the library's function, or packs its arguments.
template <typename... P, typename... A>
PyObject *finish(bool pack, pgd_status (*fn)(P...), A... a) {
  static_assert(sizeof...(P) == sizeof...(A), "arguments");
  if (pack) {
    PyObject *items[] = {to_py(a)...};
    PyObject *t = PyTuple_New(sizeof...(A));
    for (size_t i = 0; i < sizeof...(A); ++i) {
      if (!items[i] || !t) {
        Py_XDECREF(t);
        return nullptr;
      }
      PyTuple_SET_ITEM(t, i, items[i]);
    }
    return t;
  }
  pgd_status s;
  Py_BEGIN_ALLOW_THREADS
  s = fn(static_cast<P>(a)...);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong((long)s);
}

const int32_t *i32(void *p) { return static_cast<const int32_t *>(p); }
float *f32(void *p) { return static_cast<float *>(p); }

// (is_read, k_rows, v_rows, k_cache, v_cache, k_scales, v_scales, tables,
//  positions, starts or None, max_tokens or None, stream)
PyObject *range_call(PyObject *const *a) {
  Args x;
  const bool read = a[0] == Py_True;
  const at::Tensor &kr = tensor(a[1], "k rows");
  void *k_rows = x.take(a[1], at::kBFloat16, kr.sizes(), "k rows");
  void *v_rows = x.take(a[2], at::kBFloat16, kr.sizes(), "v rows");
  const auto pool = sizes(a[3], 6, "k_cache", at::kByte);
  const int64_t NB = pool[0], n_kv = pool[1], rg = pool[2];
  const auto table = sizes(a[7], 2, "block_tables");
  const int64_t B = table[0], MB = table[1];
  if (kr.dim() < 3 || kr.size(-2) != n_kv || kr.size(-1) != kDim)
    refuse(PyExc_ValueError, "rows must end in [" + std::to_string(n_kv) + "][128], got " +
                                 shape_text(kr.sizes()));
  const int64_t N = n_kv ? kr.numel() / (n_kv * kDim) : 0;
  int64_t T;
  if (a[9] == Py_None) {
    if ((N && !B) || (B && N % B))
      refuse(PyExc_ValueError,
             std::to_string(N) + " rows for " + std::to_string(B) + " sequences");
    T = B ? N / B : 0;
    if (a[10] != Py_None && integer(a[10], "max_tokens") != T)
      refuse(PyExc_ValueError, "max_tokens is not the " + std::to_string(T) +
                                   " tokens that every sequence has");
  } else if (a[10] == Py_None) {
    refuse(PyExc_ValueError, "token_starts needs max_tokens, the most tokens of a sequence");
  } else {
    T = integer(a[10], "max_tokens");
  }
  void *k = x.take(a[3], at::kByte, {NB, n_kv, rg, 8, 8, 16}, "k_cache");
  void *v = x.take(a[4], at::kByte, {NB, n_kv, rg, 8, 8, 16}, "v_cache");
  float *ks = f32(x.take(a[5], at::kFloat, {NB, n_kv}, "k_scales"));
  float *vs = f32(x.take(a[6], at::kFloat, {NB, n_kv}, "v_scales"));
  const int32_t *tables = i32(x.take(a[7], at::kInt, {B, MB}, "block_tables"));
  const int32_t *pos = i32(x.take(a[8], at::kInt, {B}, "positions"));
  const int32_t *starts = i32(x.take_opt(a[9], at::kInt, {B + 1}, "token_starts"));
  const int32_t b = int32(B, "B"), t = int32(T, "max_tokens"), n = int32(N, "rows"),
                h = int32(n_kv, "n_kv"), bs = int32(rg * 8, "block size"), mb = int32(MB, "MB"),
                nb = int32(NB, "NB");
  void *st = x.stream(a[11]);
  if (read)
    return finish(false, pgd_kv_read_fp8b, k_rows, v_rows, k, v, ks, vs, tables, pos, starts, b, t,
                  n, h, (int32_t)kDim, bs, mb, nb, st);
  return finish(false, pgd_kv_append_fp8b, k_rows, v_rows, k, v, ks, vs, tables, pos, starts, b, t,
                n, h, (int32_t)kDim, bs, mb, nb, st);
}

// (out, q, k_new or None, v_new or None, k_cache, v_cache, k_scales, v_scales,
//  tables, context_lens, scale, num_splits, workspace, stream, pack)
PyObject *attention_call(PyObject *const *a) {
  Args x;
  const auto pool = sizes(a[4], 6, "k_cache", at::kByte);
  const int64_t NB = pool[0], n_kv = pool[1], rg = pool[2];
  const auto qs = sizes(a[1], 3, "q");
  const int64_t B = qs[0], n_q = qs[1], d = qs[2];
  const int64_t MB = sizes(a[8], 2, "block_tables")[1];
  void *q = x.take(a[1], at::kBFloat16, {B, n_q, d}, "q");
  void *out = x.take(a[0], at::kBFloat16, {B, n_q, d}, "out");
  const bool append = a[2] != Py_None;
  void *kn = append ? x.take(a[2], at::kBFloat16, {B, n_kv, d}, "k_new") : nullptr;
  void *vn = append ? x.take(a[3], at::kBFloat16, {B, n_kv, d}, "v_new") : nullptr;
  void *k = x.take(a[4], at::kByte, {NB, n_kv, rg, 8, 8, 16}, "k_cache");
  void *v = x.take(a[5], at::kByte, {NB, n_kv, rg, 8, 8, 16}, "v_cache");
  float *ks = f32(x.take(a[6], at::kFloat, {NB, n_kv}, "k_scales"));
  float *vs = f32(x.take(a[7], at::kFloat, {NB, n_kv}, "v_scales"));
  const int32_t *tables = i32(x.take(a[8], at::kInt, {B, MB}, "block_tables"));
  const int32_t *ctx = i32(x.take(a[9], at::kInt, {B}, "context_lens"));
  const at::Tensor &w = tensor(a[12], "workspace");
  void *ws = x.place(w, "workspace");
  const float scale = real(a[10]);
  const int32_t splits = (int32_t)integer(a[11], "num_splits");
  const int32_t b = int32(B, "B"), nq = int32(n_q, "n_q"), h = int32(n_kv, "n_kv"),
                dd = int32(d, "d"), bs = int32(rg * 8, "block size"), mb = int32(MB, "MB"),
                nb = int32(NB, "NB");
  void *st = x.stream(a[13]);
  const bool pack = a[14] == Py_True;
  if (append)
    return finish(pack, pgd_append_decode_attention_fp8b, out, q, kn, vn, k, v, ks, vs, tables, ctx,
                  b, nq, h, dd, bs, mb, nb, scale, splits, ws, (size_t)w.nbytes(), st);
  return finish(pack, pgd_paged_decode_attention_fp8b, out, q, k, v, ks, vs, tables, ctx, b, nq, h,
                dd, bs, mb, nb, scale, splits, ws, (size_t)w.nbytes(), st);
}

// A bf16 cache, or with scales a block-scaled one.
struct Cache {
  int64_t NB, n_kv, bs;
  void *k = nullptr, *v = nullptr;
  float *ks = nullptr, *vs = nullptr;
  Cache(Args &x, PyObject *kc, PyObject *vc, PyObject *ksc, PyObject *vsc) {
    if (vc && (ksc == Py_None) != (vsc == Py_None))
      refuse(PyExc_ValueError, "a block-scaled cache needs both scales");
    const bool fp8b = ksc != Py_None;
    const auto dtype = fp8b ? at::kByte : at::kBFloat16;
    const auto pool = sizes(kc, 6, "k_cache", dtype);
    NB = pool[0];
    n_kv = pool[1];
    bs = pool[2] * 8;
    const int64_t shape[6] = {NB, n_kv, pool[2], fp8b ? 8 : 16, 8, fp8b ? 16 : 8};
    k = x.take(kc, dtype, c10::IntArrayRef(shape, 6), "k_cache");
    if (vc) v = x.take(vc, dtype, c10::IntArrayRef(shape, 6), "v_cache");
    if (fp8b) {
      ks = f32(x.take(ksc, at::kFloat, {NB, n_kv}, "k_scales"));
      if (vc) vs = f32(x.take(vsc, at::kFloat, {NB, n_kv}, "v_scales"));
    }
  }
};

// (bounds, bound_scales, k_cache, tables, context_lens, positions or None,
//  max_tokens or None, k_scales or None, stream)
PyObject *bounds_call(PyObject *const *a) {
  Args x;
  Cache c(x, a[2], nullptr, a[7], Py_None);
  const auto table = sizes(a[3], 2, "block_tables");
  const int64_t B = table[0], MB = table[1];
  int8_t *bounds =
      static_cast<int8_t *>(x.take(a[0], at::kChar, {c.NB, c.n_kv, 2, kDim}, "bounds"));
  float *scales = f32(x.take(a[1], at::kFloat, {c.NB, c.n_kv}, "bound_scales"));
  const int32_t *tables = i32(x.take(a[3], at::kInt, {B, MB}, "block_tables"));
  const int32_t *ctx = i32(x.take(a[4], at::kInt, {B}, "context_lens"));
  const int32_t *pos = i32(x.take_opt(a[5], at::kInt, {B}, "positions"));
  const int32_t T = a[6] == Py_None ? int32(MB * c.bs, "MB * block size")
                                    : (int32_t)integer(a[6], "max_tokens");
  return finish(false, pgd_block_bounds, bounds, scales, c.k, c.ks, tables, pos, ctx,
                int32(B, "B"), T, int32(c.n_kv, "n_kv"), (int32_t)kDim, int32(c.bs, "block size"),
                int32(MB, "MB"), int32(c.NB, "NB"), x.stream(a[8]));
}

// (tiles, tile_tokens, q, bounds, bound_scales, tables, context_lens,
//  keep_first, keep_last, block_size, stream)
PyObject *select_call(PyObject *const *a) {
  Args x;
  const auto bd = sizes(a[3], 4, "bounds", at::kChar);
  const int64_t NB = bd[0], n_kv = bd[1];
  const auto qs = sizes(a[2], 3, "q");
  const int64_t B = qs[0], n_q = qs[1], d = qs[2], W = sizes(a[0], 3, "tiles")[2];
  const int64_t MB = sizes(a[5], 2, "block_tables")[1];
  int32_t *tiles = static_cast<int32_t *>(x.take(a[0], at::kInt, {B, n_kv, W}, "tiles"));
  int32_t *tokens = static_cast<int32_t *>(x.take(a[1], at::kInt, {B, n_kv}, "tile_tokens"));
  void *q = x.take(a[2], at::kBFloat16, {B, n_q, d}, "q");
  int8_t *bounds = static_cast<int8_t *>(x.take(a[3], at::kChar, {NB, n_kv, 2, kDim}, "bounds"));
  float *scales = f32(x.take(a[4], at::kFloat, {NB, n_kv}, "bound_scales"));
  const int32_t *tables = i32(x.take(a[5], at::kInt, {B, MB}, "block_tables"));
  const int32_t *ctx = i32(x.take(a[6], at::kInt, {B}, "context_lens"));
  return finish(false, pgd_select_blocks, tiles, tokens, q, bounds, scales, tables, ctx,
                int32(B, "B"), int32(n_q, "n_q"), int32(n_kv, "n_kv"), int32(d, "d"),
                (int32_t)integer(a[9], "block_size"), int32(MB, "MB"), int32(NB, "NB"),
                int32(W, "W"), (int32_t)integer(a[7], "keep_first"),
                (int32_t)integer(a[8], "keep_last"), x.stream(a[10]));
}

// (out, q, k_cache, v_cache, k_scales, v_scales, bounds, bound_scales, tables,
//  context_lens, tiles, tile_tokens, keep_first, keep_last, scale, num_splits,
//  workspace, stream, pack); bounds None: the tiles are given
PyObject *tiles_call(PyObject *const *a) {
  Args x;
  Cache c(x, a[2], a[3], a[4], a[5]);
  const auto qs = sizes(a[1], 3, "q");
  const int64_t B = qs[0], n_q = qs[1], d = qs[2], W = sizes(a[10], 3, "tiles")[2];
  void *q = x.take(a[1], at::kBFloat16, {B, n_q, d}, "q");
  void *out = x.take(a[0], at::kBFloat16, {B, n_q, d}, "out");
  int32_t *tiles = static_cast<int32_t *>(x.take(a[10], at::kInt, {B, c.n_kv, W}, "tiles"));
  int32_t *tokens = static_cast<int32_t *>(x.take(a[11], at::kInt, {B, c.n_kv}, "tile_tokens"));
  const at::Tensor &w = tensor(a[16], "workspace");
  void *ws = x.place(w, "workspace");
  const float scale = real(a[14]);
  const int32_t splits = (int32_t)integer(a[15], "num_splits");
  const int32_t b = int32(B, "B"), nq = int32(n_q, "n_q"), h = int32(c.n_kv, "n_kv"),
                dd = int32(d, "d"), bs = int32(c.bs, "block size"), nb = int32(c.NB, "NB"),
                ww = int32(W, "W");
  const bool pack = a[18] == Py_True;
  if (a[6] == Py_None)
    return finish(pack, pgd_selected_decode_attention, out, q, c.k, c.v, c.ks, c.vs,
                  (const int32_t *)tiles, (const int32_t *)tokens, b, nq, h, dd, bs, nb, ww, scale,
                  splits, ws, (size_t)w.nbytes(), x.stream(a[17]));
  int8_t *bounds =
      static_cast<int8_t *>(x.take(a[6], at::kChar, {c.NB, c.n_kv, 2, kDim}, "bounds"));
  float *scales = f32(x.take(a[7], at::kFloat, {c.NB, c.n_kv}, "bound_scales"));
  const int64_t MB = sizes(a[8], 2, "block_tables")[1];
  const int32_t *tables = i32(x.take(a[8], at::kInt, {B, MB}, "block_tables"));
  const int32_t *ctx = i32(x.take(a[9], at::kInt, {B}, "context_lens"));
  return finish(pack, pgd_sparse_decode_attention, out, q, c.k, c.v, c.ks, c.vs, bounds, scales,
                tables, ctx, tiles, tokens, b, nq, h, dd, bs, int32(MB, "MB"), nb, ww,
                (int32_t)integer(a[12], "keep_first"), (int32_t)integer(a[13], "keep_last"), scale,
                splits, ws, (size_t)w.nbytes(), x.stream(a[17]));
}

// A call with its number of arguments, no C++ exception left to Python.
template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *guarded(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", n, N);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused &) {
    return nullptr;
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

#define PGD_METHOD(name, fn, n) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<fn, n>)), \
   METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    PGD_METHOD("range", range_call, 12),   PGD_METHOD("attention", attention_call, 15),
    PGD_METHOD("bounds", bounds_call, 9),  PGD_METHOD("select", select_call, 11),
    PGD_METHOD("tiles", tiles_call, 19),   {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pgd_tensors", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pgd_tensors() { return PyModule_Create(&module); }
