// tensors.cpp -- the tensor side of the binding's calls on the block-scaled and
// the 4-bit cache, on block selections, of rotary positions and of block tables
// on the GPU: checks torch tensors against the types,
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
constexpr int64_t kGroup4 = 1152;  // bytes of 16 tokens of a 4-bit tile

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
    return address(t, name);
  }
  // A tensor on the call's device: its address.
  void *address(const ::at::Tensor &t, const char *name) {
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

// The tokens of a call over ranges: rows [N] and the most of a sequence.
struct Ranges {
  int64_t N, T;
};
Ranges ranges_of(const at::Tensor &rows, int64_t n_kv, int64_t B, PyObject *starts,
                 PyObject *most) {
  if (rows.dim() < 3 || rows.size(-2) != n_kv || rows.size(-1) != kDim)
    refuse(PyExc_ValueError, "rows must end in [" + std::to_string(n_kv) + "][128], got " +
                                 shape_text(rows.sizes()));
  Ranges r;
  r.N = n_kv ? rows.numel() / (n_kv * kDim) : 0;
  if (starts == Py_None) {
    if ((r.N && !B) || (B && r.N % B))
      refuse(PyExc_ValueError,
             std::to_string(r.N) + " rows for " + std::to_string(B) + " sequences");
    r.T = B ? r.N / B : 0;
    if (most != Py_None && integer(most, "max_tokens") != r.T)
      refuse(PyExc_ValueError, "max_tokens is not the " + std::to_string(r.T) +
                                   " tokens that every sequence has");
  } else if (most == Py_None) {
    refuse(PyExc_ValueError, "token_starts needs max_tokens, the most tokens of a sequence");
  } else {
    r.T = integer(most, "max_tokens");
  }
  return r;
}

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
  const Ranges r = ranges_of(kr, n_kv, B, a[9], a[10]);
  const int64_t N = r.N, T = r.T;
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

// (is_read, k_rows, v_rows, k_cache, v_cache, tables, positions, starts or None,
//  max_tokens or None, k_scale, v_scale, stream)
PyObject *range4_call(PyObject *const *a) {
  Args x;
  const bool read = a[0] == Py_True;
  const at::Tensor &kr = tensor(a[1], "k rows");
  void *k_rows = x.take(a[1], at::kBFloat16, kr.sizes(), "k rows");
  void *v_rows = x.take(a[2], at::kBFloat16, kr.sizes(), "v rows");
  const auto pool = sizes(a[3], 4, "k_cache", at::kByte);
  const int64_t NB = pool[0], n_kv = pool[1], ng = pool[2];
  const auto table = sizes(a[5], 2, "block_tables");
  const int64_t B = table[0], MB = table[1];
  const Ranges r = ranges_of(kr, n_kv, B, a[7], a[8]);
  void *k = x.take(a[3], at::kByte, {NB, n_kv, ng, kGroup4}, "k_cache");
  void *v = x.take(a[4], at::kByte, {NB, n_kv, ng, kGroup4}, "v_cache");
  const int32_t *tables = i32(x.take(a[5], at::kInt, {B, MB}, "block_tables"));
  const int32_t *pos = i32(x.take(a[6], at::kInt, {B}, "positions"));
  const int32_t *starts = i32(x.take_opt(a[7], at::kInt, {B + 1}, "token_starts"));
  const int32_t b = int32(B, "B"), t = int32(r.T, "max_tokens"), n = int32(r.N, "rows"),
                h = int32(n_kv, "n_kv"), bs = int32(ng * 16, "block size"), mb = int32(MB, "MB"),
                nb = int32(NB, "NB");
  const float k_scale = real(a[9]), v_scale = real(a[10]);
  void *st = x.stream(a[11]);
  if (read)
    return finish(false, pgd_kv_read_fp4, k_rows, v_rows, k, v, tables, pos, starts, b, t, n, h,
                  (int32_t)kDim, bs, mb, nb, k_scale, v_scale, st);
  return finish(false, pgd_kv_append_fp4, k_rows, v_rows, k, v, tables, pos, starts, b, t, n, h,
                (int32_t)kDim, bs, mb, nb, k_scale, v_scale, st);
}

// (out, q, k_new or None, v_new or None, k_cache, v_cache, tables, context_lens,
//  scale, k_scale, v_scale, num_splits, workspace, stream, pack)
PyObject *attention4_call(PyObject *const *a) {
  Args x;
  const auto pool = sizes(a[4], 4, "k_cache", at::kByte);
  const int64_t NB = pool[0], n_kv = pool[1], ng = pool[2];
  const auto qs = sizes(a[1], 3, "q");
  const int64_t B = qs[0], n_q = qs[1], d = qs[2];
  const int64_t MB = sizes(a[6], 2, "block_tables")[1];
  void *q = x.take(a[1], at::kBFloat16, {B, n_q, d}, "q");
  void *out = x.take(a[0], at::kBFloat16, {B, n_q, d}, "out");
  const bool append = a[2] != Py_None;
  void *kn = append ? x.take(a[2], at::kBFloat16, {B, n_kv, d}, "k_new") : nullptr;
  void *vn = append ? x.take(a[3], at::kBFloat16, {B, n_kv, d}, "v_new") : nullptr;
  void *k = x.take(a[4], at::kByte, {NB, n_kv, ng, kGroup4}, "k_cache");
  void *v = x.take(a[5], at::kByte, {NB, n_kv, ng, kGroup4}, "v_cache");
  const int32_t *tables = i32(x.take(a[6], at::kInt, {B, MB}, "block_tables"));
  const int32_t *ctx = i32(x.take(a[7], at::kInt, {B}, "context_lens"));
  const at::Tensor &w = tensor(a[12], "workspace");
  void *ws = x.place(w, "workspace");
  const float scale = real(a[8]), k_scale = real(a[9]), v_scale = real(a[10]);
  const int32_t splits = (int32_t)integer(a[11], "num_splits");
  const int32_t b = int32(B, "B"), nq = int32(n_q, "n_q"), h = int32(n_kv, "n_kv"),
                dd = int32(d, "d"), bs = int32(ng * 16, "block size"), mb = int32(MB, "MB"),
                nb = int32(NB, "NB");
  void *st = x.stream(a[13]);
  const bool pack = a[14] == Py_True;
  if (append)
    return finish(pack, pgd_append_decode_attention_fp4, out, q, kn, vn, k, v, tables, ctx, b, nq,
                  h, dd, bs, mb, nb, scale, k_scale, v_scale, splits, ws, (size_t)w.nbytes(), st);
  return finish(pack, pgd_paged_decode_attention_fp4, out, q, k, v, tables, ctx, b, nq, h, dd, bs,
                mb, nb, scale, k_scale, v_scale, splits, ws, (size_t)w.nbytes(), st);
}

// Rows [T][heads][d] of bf16, strided over tokens and heads: address and
// strides (those of a dimension of one element do not matter).
void *rows_of(Args &x, PyObject *o, int64_t T, int64_t d, int64_t heads, const char *name,
              int64_t *strides) {
  const at::Tensor &t = tensor(o, name);
  if (t.scalar_type() != at::kBFloat16)
    refuse(PyExc_TypeError,
           std::string(name) + " must be torch.bfloat16, got " + dtype_name(t.scalar_type()));
  if (t.dim() != 3 || t.size(0) != T || t.size(2) != d || (heads >= 0 && t.size(1) != heads))
    refuse(PyExc_ValueError, std::string(name) + " must be [" + std::to_string(T) + "][" +
                                 (heads >= 0 ? std::to_string(heads) : "heads") + "][" +
                                 std::to_string(d) + "], got " + shape_text(t.sizes()));
  if (t.stride(2) != 1 && d != 1)
    refuse(PyExc_ValueError, std::string(name) + " must be contiguous in its last dim");
  strides[0] = t.size(0) > 1 ? t.stride(0) : 0;
  strides[1] = t.size(1) > 1 ? t.stride(1) : 0;
  return x.address(t, name);
}
// An output's elements must lie apart (a view made by expand() has one place
// for several).
void lie_apart(PyObject *o, const char *name) {
  const at::Tensor &t = tensor(o, name);
  if (t.numel() == 0) return;
  const int64_t r = t.stride(0), h = t.stride(1), T = t.size(0), n = t.size(1), d = t.size(2);
  const bool by_token = n == 1 || h >= d, heads_in_token = T == 1 || r >= (n - 1) * h + d,
             by_head = T == 1 || r >= d, tokens_in_head = n == 1 || h >= (T - 1) * r + d;
  if (!(by_token && heads_in_token) && !(by_head && tokens_in_head))
    refuse(PyExc_ValueError, std::string(name) + " has rows that overlap");
}

// (q_out, k_out or None, q, k or None, positions, frequencies, interleaved,
//  first, factor, stream)
PyObject *rope_call(PyObject *const *a) {
  Args x;
  const auto qs = sizes(a[2], 3, "q", at::kBFloat16);
  const int64_t T = qs[0], n_q = qs[1], d = qs[2];
  int64_t strides[8] = {0, 0, 0, 0, 0, 0, 0, 0}, n_kv = 0;
  void *q = rows_of(x, a[2], T, d, n_q, "q", strides + 4);
  void *q_out = rows_of(x, a[0], T, d, n_q, "q_out", strides);
  lie_apart(a[0], "q_out");
  void *k = nullptr, *k_out = nullptr;
  if (a[3] != Py_None) {
    k = rows_of(x, a[3], T, d, -1, "k", strides + 6);
    n_kv = tensor(a[3], "k").size(1);
    k_out = rows_of(x, a[1], T, d, n_kv, "k_out", strides + 2);
    lie_apart(a[1], "k_out");
  } else if (a[1] != Py_None) {
    refuse(PyExc_ValueError, "k_out without k");
  }
  const int32_t *pos = i32(x.take(a[4], at::kInt, {T}, "positions"));
  const int64_t half = sizes(a[5], 1, "frequencies")[0];
  const int64_t *freq =
      static_cast<const int64_t *>(x.take(a[5], at::kLong, {half}, "frequencies"));
  const int64_t *st = strides;
  return finish(false, pgd_rope, q_out, k_out, q, k, pos, freq, int32(T, "T"), int32(n_q, "n_q"),
                int32(n_kv, "n_kv"), int32(d, "d"), (int32_t)integer(a[7], "first"),
                int32(2 * half, "rotary"), (int32_t)(a[6] == Py_True), real(a[8]), st,
                x.stream(a[9]));
}

// (q_out, q, k, v, k_cache, v_cache, slots, positions, frequencies, interleaved,
//  first, factor, stream)
PyObject *rope_append_call(PyObject *const *a) {
  Args x;
  const auto qs = sizes(a[1], 3, "q", at::kBFloat16);
  const int64_t T = qs[0], n_q = qs[1], d = qs[2];
  const auto pool = sizes(a[4], 6, "k_cache", at::kBFloat16);
  const int64_t NB = pool[0], n_kv = pool[1], rg = pool[2];
  int64_t strides[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  void *q_out = rows_of(x, a[0], T, d, n_q, "q_out", strides);
  lie_apart(a[0], "q_out");
  void *q = rows_of(x, a[1], T, d, n_q, "q", strides + 2);
  void *k = rows_of(x, a[2], T, d, n_kv, "k", strides + 4);
  void *v = rows_of(x, a[3], T, d, n_kv, "v", strides + 6);
  void *kc = x.take(a[4], at::kBFloat16, {NB, n_kv, rg, kDim / 8, 8, 8}, "k_cache");
  void *vc = x.take(a[5], at::kBFloat16, {NB, n_kv, rg, kDim / 8, 8, 8}, "v_cache");
  const int64_t *slots = static_cast<const int64_t *>(x.take(a[6], at::kLong, {T}, "slots"));
  const int32_t *pos = i32(x.take(a[7], at::kInt, {T}, "positions"));
  const int64_t half = sizes(a[8], 1, "frequencies")[0];
  const int64_t *freq =
      static_cast<const int64_t *>(x.take(a[8], at::kLong, {half}, "frequencies"));
  const int64_t *st = strides;
  return finish(false, pgd_rope_append, q_out, q, k, v, kc, vc, slots, pos, freq, int32(T, "T"),
                int32(n_q, "n_q"), int32(n_kv, "n_kv"), int32(d, "d"), int32(rg * 8, "block size"),
                int32(NB, "NB"), (int32_t)integer(a[10], "first"), int32(2 * half, "rotary"),
                (int32_t)(a[9] == Py_True), real(a[11]), st, x.stream(a[12]));
}

int32_t *i32_out(void *p) { return static_cast<int32_t *>(p); }

// (tables, context_lens, new_tokens, refs, free_bits, block_size, positions,
//  token_starts, slots, token_positions, copy_src, copy_dst, result, stream)
PyObject *grow_call(PyObject *const *a) {
  Args x;
  const auto table = sizes(a[0], 2, "block_tables");
  const int64_t B = table[0], MB = table[1], NB = sizes(a[3], 1, "refs")[0];
  const int64_t N = sizes(a[8], 1, "slots")[0];
  int32_t *tables = i32_out(x.take(a[0], at::kInt, {B, MB}, "block_tables"));
  int32_t *ctx = i32_out(x.take(a[1], at::kInt, {B}, "context_lens"));
  const int32_t *more = i32(x.take(a[2], at::kInt, {B}, "new_tokens"));
  int32_t *refs = i32_out(x.take(a[3], at::kInt, {NB}, "refs"));
  int32_t *bits = i32_out(x.take(a[4], at::kInt, {(NB + 31) / 32}, "free_bits"));
  int32_t *pos = i32_out(x.take(a[6], at::kInt, {B}, "positions"));
  int32_t *starts = i32_out(x.take(a[7], at::kInt, {B + 1}, "token_starts"));
  int64_t *slots = static_cast<int64_t *>(x.take(a[8], at::kLong, {N}, "slots"));
  int32_t *places = i32_out(x.take(a[9], at::kInt, {N}, "token_positions"));
  int32_t *src = i32_out(x.take(a[10], at::kInt, {B}, "copy_src"));
  int32_t *dst = i32_out(x.take(a[11], at::kInt, {B}, "copy_dst"));
  int32_t *result = i32_out(x.take(a[12], at::kInt, {4}, "result"));
  return finish(false, pgd_grow_tables, tables, ctx, more, refs, bits, pos, starts, slots, places,
                src, dst, result, int32(B, "B"), int32(N, "N"),
                (int32_t)integer(a[5], "block_size"), int32(MB, "MB"), int32(NB, "NB"),
                x.stream(a[13]));
}

// (tables, context_lens, keep_lens, refs, free_bits, block_size, stream)
PyObject *trim_call(PyObject *const *a) {
  Args x;
  const auto table = sizes(a[0], 2, "block_tables");
  const int64_t B = table[0], MB = table[1], NB = sizes(a[3], 1, "refs")[0];
  int32_t *tables = i32_out(x.take(a[0], at::kInt, {B, MB}, "block_tables"));
  int32_t *ctx = i32_out(x.take(a[1], at::kInt, {B}, "context_lens"));
  const int32_t *keep = i32(x.take(a[2], at::kInt, {B}, "keep_lens"));
  int32_t *refs = i32_out(x.take(a[3], at::kInt, {NB}, "refs"));
  int32_t *bits = i32_out(x.take(a[4], at::kInt, {(NB + 31) / 32}, "free_bits"));
  return finish(false, pgd_trim_tables, tables, ctx, keep, refs, bits, int32(B, "B"),
                (int32_t)integer(a[5], "block_size"), int32(MB, "MB"), int32(NB, "NB"),
                x.stream(a[6]));
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
    PGD_METHOD("tiles", tiles_call, 19),   PGD_METHOD("range4", range4_call, 12),
    PGD_METHOD("attention4", attention4_call, 15), PGD_METHOD("rope", rope_call, 10),
    PGD_METHOD("rope_append", rope_append_call, 13), PGD_METHOD("grow", grow_call, 14),
    PGD_METHOD("trim", trim_call, 7), {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pgd_tensors", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pgd_tensors() { return PyModule_Create(&module); }
