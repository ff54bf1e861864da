// Tensor front end of the operators that a decode step calls once per linear
// or layer (fp4_quantize, fp4_linear, kv8_append, kv8_attention): the checks
// of the ctypes binding, the output allocations and the call into the C ABI
// of libw4.so, as a CPython extension, because at a few microseconds of GPU
// time per call the interpreter's share is what a user waits for (10 - 14 us
// per call through ctypes, 3 - 5 us here).  No computation happens in it.
//
// The module is loaded by __init__.py, which hands it the addresses of the C
// entry points (from the libw4.so it has loaded) and its W4Error class.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <string>

#include "w4.h"

namespace {

using at::Tensor;
using c10::IntArrayRef;
using c10::ScalarType;

decltype(&w4_fp4_quantize) p_fp4_quantize = nullptr;
decltype(&w4_fp4_linear) p_fp4_linear = nullptr;
decltype(&w4_kv8_append) p_kv8_append = nullptr;
decltype(&w4_kv8_attention) p_kv8_attention = nullptr;
PyObject* g_error_class = nullptr;  // W4Error(status, where)

// Refusals, raised as Python's TypeError and ValueError.
struct Refusal : torch::PyTorchError {
  Refusal(PyObject* t, const char* text) : PyTorchError(text), type(t) {}
  PyObject* python_type() override { return type; }
  PyObject* type;
};
__attribute__((format(printf, 1, 2))) Refusal type_error(const char* fmt, ...) {
  char text[512];
  va_list args;
  va_start(args, fmt);
  vsnprintf(text, sizeof(text), fmt, args);
  va_end(args);
  return Refusal(PyExc_TypeError, text);
}
__attribute__((format(printf, 1, 2))) Refusal value_error(const char* fmt, ...) {
  char text[512];
  va_list args;
  va_start(args, fmt);
  vsnprintf(text, sizeof(text), fmt, args);
  va_end(args);
  return Refusal(PyExc_ValueError, text);
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw type_error("%s must be a CUDA tensor", name);
  return THPVariable_Unpack(o);
}

void check_dtype(const Tensor& t, ScalarType dt, const char* name) {
  if (t.scalar_type() != dt)
    throw type_error("%s must be %s, got %s", name, c10::toString(dt),
                           c10::toString(t.scalar_type()));
}

void check_shape(const Tensor& t, IntArrayRef shape, const char* name) {
  if (t.sizes() != shape) {
    std::string want, have;
    for (int64_t v : shape) want += (want.empty() ? "" : ", ") + std::to_string(v);
    for (int64_t v : t.sizes()) have += (have.empty() ? "" : ", ") + std::to_string(v);
    throw value_error("%s has shape (%s), expected (%s)", name, have.c_str(), want.c_str());
  }
}

// A companion tensor: dtype, shape, contiguous.
const Tensor& companion(PyObject* o, ScalarType dt, IntArrayRef shape, const char* name) {
  const Tensor& t = tensor(o, name);
  check_dtype(t, dt, name);
  check_shape(t, shape, name);
  if (!t.is_contiguous()) throw value_error("%s must be contiguous", name);
  return t;
}

void check_cuda(const Tensor& t, const char* name) {
  if (!t.is_cuda()) throw type_error("%s must be a CUDA tensor", name);
}

// The kernels run on one device and write through every pointer they get.
void check_device(const Tensor& t, const c10::Device& at, const char* name) {
  if (t.device() != at)
    throw value_error("%s is on %s, the call runs on %s", name, t.device().str().c_str(),
                            at.str().c_str());
}

// Elements between the rows (first axis) of a tensor whose rows are
// contiguous: slices of a wider buffer's rows are allowed.
int64_t row_stride(const Tensor& t, const char* name) {
  int64_t inner = 1;
  for (int64_t d = t.dim() - 1; d > 0; --d) {
    if (t.size(d) != 1 && t.stride(d) != inner)
      throw value_error("%s: only the first axis may be strided", name);
    inner *= t.size(d);
  }
  if (t.size(0) <= 1) return inner;
  if (t.stride(0) < inner) throw value_error("%s: rows overlap", name);
  return t.stride(0);
}

Tensor empty(IntArrayRef shape, ScalarType dt, const c10::Device& at) {
  return at::detail::empty_cuda(shape, dt, at, std::nullopt);
}

void* stream_of(const c10::Device& at) {
  return c10::cuda::getCurrentCUDAStream(at.index()).stream();
}

// "mx" / "nv" -> format, channels per block.
int fp4_format(PyObject* o, int64_t* block) {
  const char* s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
  if (s && s[0] == 'm' && s[1] == 'x' && !s[2]) return *block = 32, W4_FP4_MX;
  if (s && s[0] == 'n' && s[1] == 'v' && !s[2]) return *block = 16, W4_FP4_NV;
  PyErr_Clear();
  throw value_error("format must be 'mx' or 'nv'");
}

int64_t integer(PyObject* o, const char* name) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw type_error("%s must be an integer", name);
  }
  return v;
}

void check_status(w4_status st, const char* where) {
  if (st == W4_OK) return;
  PyObject* e = PyObject_CallFunction(g_error_class, "is", static_cast<int>(st), where);
  if (e) {
    PyErr_SetObject(g_error_class, e);
    Py_DECREF(e);
  }
  throw python_error();
}

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }
PyObject* wrap_or_none(const Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}

#define NARGS(n, what) \
  if (nargs != n) throw type_error(what " takes %d arguments", n)

// init(fp4_quantize, fp4_linear, kv8_append, kv8_attention, W4Error)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  NARGS(5, "init");
  p_fp4_quantize = reinterpret_cast<decltype(p_fp4_quantize)>(PyLong_AsVoidPtr(a[0]));
  p_fp4_linear = reinterpret_cast<decltype(p_fp4_linear)>(PyLong_AsVoidPtr(a[1]));
  p_kv8_append = reinterpret_cast<decltype(p_kv8_append)>(PyLong_AsVoidPtr(a[2]));
  p_kv8_attention = reinterpret_cast<decltype(p_kv8_attention)>(PyLong_AsVoidPtr(a[3]));
  if (PyErr_Occurred()) throw python_error();
  Py_INCREF(a[4]);
  g_error_class = a[4];
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// fp4_quantize(x, fmt, values)
PyObject* fp4_quantize(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  NARGS(3, "fp4_quantize");
  int64_t block = 0;
  const int fmt = fp4_format(a[1], &block);
  const int with_values = PyObject_IsTrue(a[2]);
  if (with_values < 0) throw python_error();
  const Tensor& x = tensor(a[0], "x");
  check_dtype(x, ScalarType::BFloat16, "x");
  if (x.dim() != 2) throw value_error("x must be [R, K]");
  const int64_t r = x.size(0), k = x.size(1), ldx = row_stride(x, "x");
  check_cuda(x, "x");
  const c10::Device at = x.device();
  const c10::cuda::CUDAGuard guard(at);
  const Tensor codes = empty({r, k / 2}, ScalarType::Byte, at);
  const Tensor scales = empty({(r + 127) / 128, k / (4 * block), 512}, ScalarType::Byte, at);
  Tensor row, values;
  if (fmt == W4_FP4_NV) row = empty({r}, ScalarType::Float, at);
  if (with_values) values = empty({r, k}, ScalarType::BFloat16, at);
  check_status(p_fp4_quantize(x.data_ptr(), r, k, ldx, fmt,
                              static_cast<uint8_t*>(codes.data_ptr()),
                              static_cast<uint8_t*>(scales.data_ptr()),
                              row.defined() ? static_cast<float*>(row.data_ptr()) : nullptr,
                              values.defined() ? values.data_ptr() : nullptr, stream_of(at)),
               "w4_fp4_quantize");
  PyObject* out = PyTuple_New(with_values ? 4 : 3);
  PyTuple_SET_ITEM(out, 0, wrap(codes));
  PyTuple_SET_ITEM(out, 1, wrap(scales));
  PyTuple_SET_ITEM(out, 2, wrap_or_none(row));
  if (with_values) PyTuple_SET_ITEM(out, 3, wrap(values));
  return out;
  END_HANDLE_TH_ERRORS
}

// fp4_linear(xcodes, xscales, xrow, wcodes, wscales, wrow, fmt, flags, out)
PyObject* fp4_linear(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  NARGS(9, "fp4_linear");
  int64_t block = 0;
  const int fmt = fp4_format(a[6], &block);
  const Tensor& xc = tensor(a[0], "xcodes");
  const Tensor& wc = tensor(a[3], "wcodes");
  check_dtype(xc, ScalarType::Byte, "xcodes");
  if (xc.dim() != 2 || wc.dim() != 2)
    throw value_error("xcodes and wcodes must be [rows, K/2]");
  if (!xc.is_contiguous()) throw value_error("xcodes must be contiguous");
  const int64_t m = xc.size(0), k2 = xc.size(1), n = wc.size(0), tiles = 2 * k2 / (4 * block);
  companion(a[3], ScalarType::Byte, {n, k2}, "wcodes");
  const Tensor& xs = companion(a[1], ScalarType::Byte, {(m + 127) / 128, tiles, 512}, "xscales");
  const Tensor& ws = companion(a[4], ScalarType::Byte, {(n + 127) / 128, tiles, 512}, "wscales");
  const bool nv = fmt == W4_FP4_NV;
  if ((a[2] == Py_None) == nv || (a[5] == Py_None) == nv)
    throw value_error("xrow and wrow belong to format 'nv' alone");
  Tensor xr, wr, y;
  if (nv) {
    xr = companion(a[2], ScalarType::Float, {m}, "xrow");
    wr = companion(a[5], ScalarType::Float, {n}, "wrow");
  }
  const int64_t flags = integer(a[7], "flags");
  if (a[8] != Py_None) y = companion(a[8], ScalarType::BFloat16, {m, n}, "out");
  check_cuda(xc, "xcodes");
  const c10::Device at = xc.device();
  check_device(xs, at, "xscales");
  check_device(wc, at, "wcodes");
  check_device(ws, at, "wscales");
  if (nv) {
    check_device(xr, at, "xrow");
    check_device(wr, at, "wrow");
  }
  if (y.defined()) check_device(y, at, "out");
  const c10::cuda::CUDAGuard guard(at);
  if (!y.defined()) y = empty({m, n}, ScalarType::BFloat16, at);
  check_status(
      p_fp4_linear(static_cast<const uint8_t*>(xc.data_ptr()),
                   static_cast<const uint8_t*>(xs.data_ptr()),
                   nv ? static_cast<const float*>(xr.data_ptr()) : nullptr, m,
                   static_cast<const uint8_t*>(wc.data_ptr()),
                   static_cast<const uint8_t*>(ws.data_ptr()),
                   nv ? static_cast<const float*>(wr.data_ptr()) : nullptr, n, 2 * k2, fmt,
                   y.data_ptr(), flags < 0 || flags > 0x7FFFFFFF ? ~0u : static_cast<unsigned>(flags),
                   stream_of(at)),
      "w4_fp4_linear");
  return wrap(y);
  END_HANDLE_TH_ERRORS
}

// What appending and attention share.
struct CacheArgs {
  w4_kv8_cache c;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* starts;
  int64_t batch, max_pages, max_new;
};

// a: cache (k_codes, v_codes, k_scales, v_scales), page_table, seq_lens,
// starts or None, max_new or None; ref: the new tokens [rows, heads, d], with
// the cache's heads where kv_heads.
CacheArgs cache_args(PyObject* cache, PyObject* o_table, PyObject* o_lens, PyObject* o_starts,
                     PyObject* o_most, const Tensor& ref, const char* ref_name, bool kv_heads) {
  if (!PyTuple_Check(cache) || PyTuple_GET_SIZE(cache) != 4)
    throw type_error("cache must be a KV8Cache");
  const Tensor& k = tensor(PyTuple_GET_ITEM(cache, 0), "k_codes");
  const ScalarType dt = k.scalar_type();
  if (dt != ScalarType::Char && dt != ScalarType::Float8_e4m3fn)
    throw type_error("cache codes must be int8 or float8_e4m3fn");
  if (k.dim() != 4)
    throw value_error("k_codes must be [pages, kv_heads, page_size, head_dim]");
  if (!k.is_contiguous()) throw value_error("k_codes must be contiguous");
  const int64_t pages = k.size(0), heads = k.size(1), page = k.size(2), d = k.size(3);
  const Tensor& v = companion(PyTuple_GET_ITEM(cache, 1), dt, {pages, heads, d, page}, "v_codes");
  const Tensor& ks = companion(PyTuple_GET_ITEM(cache, 2), ScalarType::Float, {pages, heads},
                               "k_scales");
  const Tensor& vs = companion(PyTuple_GET_ITEM(cache, 3), ScalarType::Float, {pages, heads},
                               "v_scales");
  const Tensor& table = tensor(o_table, "page_table");
  check_dtype(table, ScalarType::Int, "page_table");
  if (table.dim() != 2) throw value_error("page_table must be [batch, max_pages]");
  if (!table.is_contiguous()) throw value_error("page_table must be contiguous");
  const int64_t b = table.size(0);
  const Tensor& lens = companion(o_lens, ScalarType::Int, {b}, "seq_lens");
  Tensor starts;
  int64_t most = 1;
  if (o_starts != Py_None) {
    starts = companion(o_starts, ScalarType::Int, {b + 1}, "starts");
    if (o_most == Py_None) throw value_error("max_new is needed with starts");
    most = integer(o_most, "max_new");
  } else if (o_most != Py_None && integer(o_most, "max_new") != 1) {
    throw value_error("without starts every sequence has one new token");
  }
  if (ref.dim() != 3 || ref.size(2) != d)
    throw value_error("new tokens must be [rows, heads, %ld]", static_cast<long>(d));
  if (kv_heads && ref.size(1) != heads)
    throw value_error("%s has %ld heads, the cache %ld", ref_name, static_cast<long>(ref.size(1)),
                      static_cast<long>(heads));
  if (pages > 0x7FFFFFFF || heads > 0x7FFFFFFF || page > 0x7FFFFFFF || d > 0x7FFFFFFF)
    throw value_error("cache too large");
  check_cuda(ref, ref_name);
  const c10::Device at = ref.device();
  check_device(k, at, "k_codes");
  check_device(v, at, "v_codes");
  check_device(ks, at, "k_scales");
  check_device(vs, at, "v_scales");
  check_device(table, at, "page_table");
  check_device(lens, at, "seq_lens");
  if (starts.defined()) check_device(starts, at, "starts");
  CacheArgs r;
  r.c = w4_kv8_cache{k.data_ptr(), v.data_ptr(), static_cast<float*>(ks.data_ptr()),
                     static_cast<float*>(vs.data_ptr()), static_cast<int32_t>(pages),
                     static_cast<int32_t>(heads), static_cast<int32_t>(page),
                     static_cast<int32_t>(d),
                     dt == ScalarType::Char ? W4_KV8_INT8 : W4_KV8_E4M3};
  r.table = static_cast<const int32_t*>(table.data_ptr());
  r.lens = static_cast<const int32_t*>(lens.data_ptr());
  r.starts = starts.defined() ? static_cast<const int32_t*>(starts.data_ptr()) : nullptr;
  r.batch = b;
  r.max_pages = table.size(1);
  r.max_new = most;
  return r;
}

// kv8_append(cache, k, v, page_table, seq_lens, starts, max_new)
PyObject* kv8_append(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  NARGS(7, "kv8_append");
  const Tensor& k = tensor(a[1], "k");
  const Tensor& v = tensor(a[2], "v");
  check_dtype(k, ScalarType::BFloat16, "k");
  check_dtype(v, ScalarType::BFloat16, "v");
  if (k.dim() != 3) throw value_error("k must be [rows, kv_heads, head_dim]");
  check_shape(v, k.sizes(), "v");
  const int64_t ldk = row_stride(k, "k"), ldv = row_stride(v, "v");
  const CacheArgs c = cache_args(a[0], a[3], a[4], a[5], a[6], k, "k", true);
  const c10::Device at = k.device();
  check_device(v, at, "v");
  const c10::cuda::CUDAGuard guard(at);
  check_status(p_kv8_append(&c.c, k.data_ptr(), ldk, v.data_ptr(), ldv, k.size(0), c.table,
                            c.max_pages, c.lens, c.starts, c.batch, c.max_new, stream_of(at)),
               "w4_kv8_append");
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// kv8_attention(q, cache, page_table, seq_lens, starts, max_new, scale, out)
PyObject* kv8_attention(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  NARGS(8, "kv8_attention");
  const Tensor& q = tensor(a[0], "q");
  check_dtype(q, ScalarType::BFloat16, "q");
  if (q.dim() != 3) throw value_error("q must be [rows, q_heads, head_dim]");
  const int64_t ldq = row_stride(q, "q");
  Tensor out;
  if (a[7] != Py_None) out = companion(a[7], ScalarType::BFloat16, q.sizes(), "out");
  const CacheArgs c = cache_args(a[1], a[2], a[3], a[4], a[5], q, "q", false);
  const c10::Device at = q.device();
  if (out.defined()) check_device(out, at, "out");
  double scale;
  if (a[6] == Py_None) {
    scale = c.c.head_dim == 64 ? 0.125 : 0.08838834764831845;  // 1 / sqrt(64), 1 / sqrt(128)
  } else {
    scale = PyFloat_AsDouble(a[6]);
    if (PyErr_Occurred()) throw python_error();
  }
  const c10::cuda::CUDAGuard guard(at);
  if (!out.defined()) out = empty(q.sizes(), ScalarType::BFloat16, at);
  check_status(p_kv8_attention(q.data_ptr(), ldq, q.size(0), q.size(1), &c.c, c.table, c.max_pages,
                               c.lens, c.starts, c.batch, c.max_new, static_cast<float>(scale),
                               out.data_ptr(), stream_of(at)),
               "w4_kv8_attention");
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))

PyMethodDef methods[] = {
    {"init", FAST(init), METH_FASTCALL, nullptr},
    {"fp4_quantize", FAST(fp4_quantize), METH_FASTCALL, nullptr},
    {"fp4_linear", FAST(fp4_linear), METH_FASTCALL, nullptr},
    {"kv8_append", FAST(kv8_append), METH_FASTCALL, nullptr},
    {"kv8_attention", FAST(kv8_attention), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors(void) { return PyModule_Create(&module); }
