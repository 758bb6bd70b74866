// Host path of the generation operators for Python: argument checks and the
// call of the C ABI, on torch's tensors.
//
// A step of generation is a few microseconds of kernels per call.  The same
// checks written in Python, with the call through ctypes, take 7 to 11 us a
// call, more than the kernels; here they take well under one.  The module
// holds no state besides what bind() gives it, and computes nothing.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <string>

#include "../../include/h3attn.h"

namespace {

PyObject* g_error = nullptr;     // H3AttnError(status, where)
PyObject* g_paged_kv = nullptr;  // PagedKV
PyObject *s_address, *s_device, *s_cuda_stream;

struct Entry {
  decltype(&h3attn_add_rmsnorm) add_rmsnorm;
  decltype(&h3attn_rope_table) rope_table;
  decltype(&h3attn_qk_norm_rope_append) append;
  decltype(&h3attn_paged_decode) decode;
} g_entry;

// An argument that is refused; status 0: a Python error is set already.
struct Refused {
  int status;
  std::string what;
};
[[noreturn]] void refuse(const std::string& what) { throw Refused{H3ATTN_ERR_INVALID_ARG, what}; }
[[noreturn]] void python_error() { throw Refused{0, ""}; }

const at::Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
const at::Tensor* maybe(const char* name, PyObject* o) { return o == Py_None ? nullptr : &tensor(name, o); }

std::string of_kind(at::IntArrayRef shape, at::ScalarType type) {
  std::ostringstream s;
  s << "[";
  for (size_t i = 0; i < shape.size(); ++i) s << (i ? ", " : "") << shape[i];
  s << "] " << at::toString(type) << " CUDA tensor";
  return s.str();
}
// The device of t, which has to be the current one: the library launches there.
int current_device(const char* name, const at::Tensor& t) {
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  if (t.get_device() != c10::cuda::current_device()) refuse(std::string(name) + " must be on the current device");
  return static_cast<int>(t.get_device());
}
void check_rest(const char* name, const at::Tensor& t, int dev) {
  if (t.requires_grad()) refuse(std::string(name) + ": inference only, grad-enabled inputs are rejected");
  if (t.get_device() != dev) refuse(std::string(name) + " must be on the current device");
}
// A contiguous tensor of this type and shape on device dev, without a gradient.
void check(const char* name, const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape, int dev) {
  if (t.scalar_type() != type || !t.is_cuda() || !t.is_contiguous() || t.sizes() != shape)
    refuse(std::string(name) + " must be a contiguous " + of_kind(shape, type));
  check_rest(name, t, dev);
}
template <class T>
const T* data(const at::Tensor* t) {
  return t ? static_cast<const T*>(t->const_data_ptr()) : nullptr;
}
template <class T>
const T* checked(const char* name, const at::Tensor* t, at::ScalarType type, at::IntArrayRef shape, int dev) {
  if (!t) return nullptr;
  check(name, *t, type, shape, dev);
  return data<T>(t);
}

// Elements from one token to the next of a [B, S, H, D] bf16 tensor whose heads
// lie behind one another (a slice of a fused projection, say).
int64_t token_stride(const char* name, const at::Tensor& t, int64_t B, int64_t S, int64_t H, int64_t D, int dev) {
  const int64_t shape[] = {B, S, H, D};
  if (t.scalar_type() != at::kBFloat16 || !t.is_cuda() || t.sizes() != at::IntArrayRef(shape, 4))
    refuse(std::string(name) + " must be a " + of_kind({shape, 4}, at::kBFloat16));
  check_rest(name, t, dev);
  if (B * S * H == 0) return H * D;
  const int64_t sb = t.stride(0), ss = t.stride(1), sh = t.stride(2), sd = t.stride(3);
  if (sd != 1 || (H > 1 && sh != D) || (S > 1 && B > 1 && sb != S * ss))
    refuse(std::string(name) + " must have contiguous heads and one stride from token to token");
  return S > 1 ? ss : B > 1 ? sb : H * D;
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) python_error();
  return v;
}
int int32(const char* name, PyObject* o) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " must fit 32 bits");
  return static_cast<int>(v);
}
int int32(const char* name, int64_t v) {
  if (v > INT32_MAX) refuse(std::string(name) + " must fit 32 bits");
  return static_cast<int>(v);
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) python_error();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) python_error();
  return v != 0;
}
int64_t attribute(PyObject* o, PyObject* name) {
  PyObject* v = PyObject_GetAttr(o, name);
  if (!v) python_error();
  const int64_t n = PyLong_AsLongLong(v);
  Py_DECREF(v);
  if (n == -1 && PyErr_Occurred()) python_error();
  return n;
}
// None: the current stream of device dev; a handle; or an object with cuda_stream.
h3attn_stream_t stream_of(PyObject* o, int dev) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  if (PyLong_Check(o)) return reinterpret_cast<h3attn_stream_t>(static_cast<intptr_t>(integer(o)));
  return reinterpret_cast<h3attn_stream_t>(static_cast<intptr_t>(attribute(o, s_cuda_stream)));
}
// The descriptor that a PagedKV keeps.
const h3attn_paged_kv_t& cache_of(PyObject* o, int dev) {
  const int is = PyObject_IsInstance(o, g_paged_kv);
  if (is < 0) python_error();
  if (!is) refuse("cache must be a PagedKV");
  if (attribute(o, s_device) != dev) refuse("the cache must be on the current device");
  return *reinterpret_cast<const h3attn_paged_kv_t*>(static_cast<intptr_t>(attribute(o, s_address)));
}

void raise(int status, const char* where) {
  PyObject* e = PyObject_CallFunction(g_error, "is", status, where);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
}
// Runs body() -> status and turns what goes wrong into a Python error.
template <class F>
PyObject* guarded(const char* where, PyObject* result, F&& body) {
  try {
    if (!g_error) refuse("the library is not loaded");
    const h3attn_status_t st = body();
    if (st == H3ATTN_OK) {
      Py_INCREF(result);
      return result;
    }
    raise(st, where);
  } catch (const Refused& r) {
    if (r.status) raise(r.status, r.what.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, where);
  }
  return nullptr;
}
template <class F>
h3attn_status_t without_gil(F&& call) {
  PyThreadState* state = PyEval_SaveThread();
  const h3attn_status_t st = call();
  PyEval_RestoreThread(state);
  return st;
}
bool count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) PyErr_Format(PyExc_TypeError, "%zd arguments, got %zd", want, n);
  return n == want;
}

// x, residual, h, y, w, eps, y_scale, stream
PyObject* add_rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 8)) return nullptr;
  return guarded("h3attn_add_rmsnorm", a[3], [&] {
    const at::Tensor &x = tensor("x", a[0]), &y = tensor("y", a[3]);
    const at::Tensor *residual = maybe("residual", a[1]), *h = maybe("h", a[2]), *w = maybe("w", a[4]),
                     *y_scale = maybe("y_scale", a[6]);
    const int dev = current_device("x", x);
    if (x.dim() != 2) refuse("x must be a [T, C] bf16 CUDA tensor");
    const at::IntArrayRef shape = x.sizes();
    const int T = int32("T", shape[0]), C = int32("C", shape[1]);
    check("x", x, at::kBFloat16, shape, dev);
    if (!residual != !h) refuse("residual and h must be given together");
    checked<void>("residual", residual, at::kBFloat16, shape, dev);
    checked<void>("h", h, at::kBFloat16, shape, dev);
    const float* wp = checked<float>("w", w, at::kFloat, {C}, dev);
    int format = H3ATTN_Y_BF16;
    if (y.scalar_type() == at::kBFloat16) {
      if (y_scale) refuse("a bf16 y takes no y_scale");
      check("y", y, at::kBFloat16, shape, dev);
    } else {
      check("y", y, at::kFloat8_e4m3fn, shape, dev);
      if (!y_scale) refuse("an e4m3 y needs y_scale");
      if (y_scale->scalar_type() == at::kFloat) {
        check("y_scale", *y_scale, at::kFloat, {T}, dev);
        format = H3ATTN_Y_E4M3_ROW;
      } else {
        check("y_scale", *y_scale, y_scale->scalar_type() == at::kByte ? at::kByte : at::kFloat8_e8m0fnu, {T, C / 32}, dev);
        format = H3ATTN_Y_E4M3_MX32;
      }
    }
    const float eps = static_cast<float>(number(a[5]));
    const h3attn_stream_t s = stream_of(a[7], dev);
    return without_gil([&] {
      return g_entry.add_rmsnorm(data<void>(&x), data<void>(residual), const_cast<void*>(data<void>(h)),
                                 const_cast<void*>(data<void>(&y)), wp, const_cast<void*>(data<void>(y_scale)), T, C, format,
                                 eps, s);
    });
  });
}

// cos, sin, rotary_dim, theta, address of the scaling or 0, pos, first, stream
PyObject* rope_table(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 8)) return nullptr;
  return guarded("h3attn_rope_table", Py_None, [&] {
    const at::Tensor &cos = tensor("cos", a[0]), &sin = tensor("sin", a[1]);
    const at::Tensor* pos = maybe("pos", a[5]);
    const int dev = current_device("cos", cos), rotary_dim = int32("rotary_dim", a[2]);
    const int N = int32("N", cos.dim() > 0 ? cos.size(0) : 0);
    check("cos", cos, at::kFloat, {N, rotary_dim / 2}, dev);
    check("sin", sin, at::kFloat, {N, rotary_dim / 2}, dev);
    const int32_t* pp = checked<int32_t>("pos", pos, at::kInt, {N}, dev);
    const double theta = number(a[3]);
    const auto* scaling = reinterpret_cast<const h3attn_rope_scaling_t*>(static_cast<intptr_t>(integer(a[4])));
    const int64_t first = integer(a[6]);
    const h3attn_stream_t s = stream_of(a[7], dev);
    return without_gil([&] {
      return g_entry.rope_table(const_cast<float*>(data<float>(&cos)), const_cast<float*>(data<float>(&sin)), pp, first, N,
                                rotary_dim, theta, scaling, s);
    });
  });
}

// q, k, v, q_out, cache, wq, wk, cos, sin, rotary_dim, eps, interleaved, pos, new_len, len_out, stream
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 16)) return nullptr;
  return guarded("h3attn_qk_norm_rope_append", a[3], [&] {
    const at::Tensor *q = maybe("q", a[0]), *q_out = maybe("q_out", a[3]), *wq = maybe("wq", a[5]), *wk = maybe("wk", a[6]),
                     *cos = maybe("cos", a[7]), *sin = maybe("sin", a[8]), *pos = maybe("pos", a[12]),
                     *new_len = maybe("new_len", a[13]), *len_out = maybe("len_out", a[14]);
    const at::Tensor &k = tensor("k", a[1]), &v = tensor("v", a[2]);
    const int dev = current_device("k", k);
    const h3attn_paged_kv_t& cache = cache_of(a[4], dev);
    const int64_t B = cache.B, Hkv = cache.Hkv, D = cache.D;
    if (k.dim() != 4) refuse("k must be a [B, S, Hkv, D] bf16 CUDA tensor");
    const int S = int32("S", k.size(1));
    const int64_t ks = token_stride("k", k, B, S, Hkv, D, dev), vs = token_stride("v", v, B, S, Hkv, D, dev);
    int Hq = 0;
    int64_t qs = 0;
    if (!q != !q_out) refuse("q_out must be given exactly when q is");
    if (q) {
      if (q->dim() != 4) refuse("q must be a [B, S, Hq, D] bf16 CUDA tensor");
      Hq = int32("Hq", q->size(2));
      qs = token_stride("q", *q, B, S, Hq, D, dev);
      check("q_out", *q_out, at::kBFloat16, {B, S, Hq, D}, dev);
    }
    const float* wqp = checked<float>("wq", wq, at::kFloat, {D}, dev);
    const float* wkp = checked<float>("wk", wk, at::kFloat, {D}, dev);
    const int rotary_dim = int32("rotary_dim", a[9]);
    int rows = 0;
    const float *cp = nullptr, *sp = nullptr;
    if (rotary_dim > 0) {
      if (!cos || !sin) refuse("cos and sin are required when rotary_dim > 0");
      rows = int32("rows", cos->dim() > 0 ? cos->size(0) : 0);
      cp = checked<float>("cos", cos, at::kFloat, {rows, rotary_dim / 2}, dev);
      sp = checked<float>("sin", sin, at::kFloat, {rows, rotary_dim / 2}, dev);
    }
    const int32_t* pp = checked<int32_t>("pos", pos, at::kInt, {B, S}, dev);
    const int32_t* np = checked<int32_t>("new_len", new_len, at::kInt, {B}, dev);
    const int32_t* lp = checked<int32_t>("len_out", len_out, at::kInt, {B}, dev);
    const float eps = static_cast<float>(number(a[10]));
    const int interleaved = truth(a[11]) ? 1 : 0;
    const h3attn_stream_t s = stream_of(a[15], dev);
    return without_gil([&] {
      return g_entry.append(data<void>(q), data<void>(&k), data<void>(&v), const_cast<void*>(data<void>(q_out)), &cache, wqp, wkp,
                            cp, sp, pp, np, const_cast<int32_t*>(lp), S, Hq, qs, ks, vs, rows, rotary_dim, interleaved, eps, s);
    });
  });
}

// q, o, cache, scale or None, workspace, stream
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 6)) return nullptr;
  return guarded("h3attn_paged_decode", a[1], [&] {
    const at::Tensor &q = tensor("q", a[0]), &o = tensor("o", a[1]);
    const at::Tensor* workspace = maybe("workspace", a[4]);
    const int dev = current_device("q", q);
    const h3attn_paged_kv_t& cache = cache_of(a[2], dev);
    const at::IntArrayRef shape = q.sizes();
    if (!(shape.size() == 3 || (shape.size() == 4 && shape[1] == 1)))
      refuse("q must be [B, 1, Hq, D] or [B, Hq, D]: one new token per sequence");
    const int Hq = int32("Hq", shape[shape.size() - 2]);
    if (shape[0] != cache.B || shape.back() != cache.D) refuse("shape mismatch between q and the cache");
    check("q", q, at::kBFloat16, shape, dev);
    check("o", o, at::kBFloat16, shape, dev);
    size_t bytes = 0;
    if (workspace) {
      if (!workspace->is_cuda() || workspace->get_device() != dev || !workspace->is_contiguous())
        refuse("workspace must be a contiguous CUDA tensor on the current device");
      bytes = workspace->nbytes();
    }
    const float scale = a[3] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(cache.D)))
                                        : static_cast<float>(number(a[3]));
    const h3attn_stream_t s = stream_of(a[5], dev);
    return without_gil([&] {
      return g_entry.decode(data<void>(&q), const_cast<void*>(data<void>(&o)), &cache, Hq, scale,
                            const_cast<void*>(data<void>(workspace)), bytes, s);
    });
  });
}

// H3AttnError, PagedKV, and the addresses of the four entry points of the loaded library
PyObject* bind(PyObject*, PyObject* args) {
  PyObject *error, *paged_kv;
  unsigned long long at[4];
  if (!PyArg_ParseTuple(args, "OOKKKK", &error, &paged_kv, &at[0], &at[1], &at[2], &at[3])) return nullptr;
  Py_INCREF(error);
  Py_INCREF(paged_kv);
  Py_XDECREF(g_error);
  Py_XDECREF(g_paged_kv);
  g_error = error;
  g_paged_kv = paged_kv;
  g_entry.add_rmsnorm = reinterpret_cast<decltype(g_entry.add_rmsnorm)>(at[0]);
  g_entry.rope_table = reinterpret_cast<decltype(g_entry.rope_table)>(at[1]);
  g_entry.append = reinterpret_cast<decltype(g_entry.append)>(at[2]);
  g_entry.decode = reinterpret_cast<decltype(g_entry.decode)>(at[3]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef g_methods[] = {method<add_rmsnorm>("add_rmsnorm"), method<rope_table>("rope_table"), method<append>("append"),
                           method<decode>("decode"), {"bind", bind, METH_VARARGS, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_step", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__step() {
  s_address = PyUnicode_InternFromString("_address");
  s_device = PyUnicode_InternFromString("_device");
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  return s_address && s_device && s_cuda_stream ? PyModule_Create(&g_module) : nullptr;
}
