// pycall.cpp -- argument checks and the C calls of the device-planned serving
// operators, for vpp.py.  Their kernels take a few microseconds at decode sizes,
// less than ctypes takes to convert thirty arguments, or Python's attribute calls to
// read ten tensors (an append: 24.7 us of host time by ctypes, 6.8 us through attribute
// calls from C, 2.8 us here; a decode call 23.5, 8.9 and 5.4 us); here the tensors'
// own fields are read and the library's functions called by address.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>

#include "vpp.h"

namespace {

decltype(&vpp_rope_append) f_rope;
decltype(&vpp_rope_append_fp8) f_rope_fp8;
decltype(&vpp_decode_attn) f_decode;
decltype(&vpp_decode_attn_fp8) f_decode_fp8;
decltype(&vpp_prompt_attn) f_prompt;

struct Refused {};  // a Python error is set

template <typename... A>
[[noreturn]] void refuse(const char* format, A... a) {
  PyErr_Format(PyExc_ValueError, format, a...);
  throw Refused{};
}

void check_python() {
  if (PyErr_Occurred()) throw Refused{};
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor", what);
    throw Refused{};
  }
  return THPVariable_Unpack(o);
}

// A tensor of `dims` dimensions.
const at::Tensor& of_dims(PyObject* o, int dims, const char* what) {
  const at::Tensor& t = tensor(o, what);
  if (t.dim() != dims) refuse("%s must have %d dimensions, not %lld", what, dims, static_cast<long long>(t.dim()));
  return t;
}

// Type and device (a negative `dev` takes host tensors, for tests of these checks).
void check_kind(const at::Tensor& t, at::ScalarType type, long dev, const char* what) {
  if (t.scalar_type() != type) refuse("%s must be %s", what, c10::toString(type));
  if (t.get_device() != dev || t.is_cuda() != (dev >= 0)) refuse("%s must be on the current CUDA device", what);
}

// Address of a contiguous tensor of this type and shape.
template <int N>
void* array(PyObject* o, at::ScalarType type, long dev, const int64_t (&shape)[N], const char* what) {
  const at::Tensor& t = of_dims(o, N, what);
  check_kind(t, type, dev, what);
  for (int i = 0; i < N; ++i)
    if (t.size(i) != shape[i])
      refuse("%s has the wrong shape: dimension %d is %lld, not %lld", what, i, static_cast<long long>(t.size(i)),
             static_cast<long long>(shape[i]));
  if (!t.is_contiguous()) refuse("%s must be contiguous", what);
  return t.data_ptr();
}

// A bf16 [n, h, d] tensor whose heads are contiguous within a token (a part of a
// wider projection is): address and token stride.  The stride of a single token is
// never used and reported as the row's length.
struct Rows {
  void* p = nullptr;
  int64_t stride = 0;
  Rows() = default;
  Rows(PyObject* o, long dev, int64_t n, int64_t h, int64_t d, const char* what) {
    const at::Tensor& t = of_dims(o, 3, what);
    check_kind(t, at::kBFloat16, dev, what);
    if (t.size(0) != n || t.size(1) != h || t.size(2) != d)
      refuse("%s must be [%lld, %lld, %lld], not [%lld, %lld, %lld]", what, static_cast<long long>(n),
             static_cast<long long>(h), static_cast<long long>(d), static_cast<long long>(t.size(0)),
             static_cast<long long>(t.size(1)), static_cast<long long>(t.size(2)));
    stride = h * d;
    if (!t.is_contiguous()) {
      if ((t.stride(2) != 1 && d > 1) || (t.stride(1) != d && h > 1))
        refuse("%s: a token's heads must be contiguous", what);
      if (n > 1) stride = t.stride(0);
    }
    p = t.data_ptr();
  }
};

// A paged cache: blocks, kv heads, dims and addresses.
struct Cache {
  int64_t nb, hkv, dq, dv;
  void *k, *v;
  Cache(PyObject* key, PyObject* value, bool fp8, long dev) {
    const at::Tensor &tk = of_dims(key, 4, "k_cache"), &tv = of_dims(value, 4, "v_cache");
    nb = tk.size(0);
    hkv = tk.size(2);
    dq = tk.size(3);
    dv = tv.size(3);
    const at::ScalarType type = fp8 ? at::kByte : at::kBFloat16;
    const int64_t ks[4] = {nb, 64, hkv, dq}, vs[4] = {nb, 64, hkv, dv};
    k = array(key, type, dev, ks, "k_cache");
    v = array(value, type, dev, vs, "v_cache");
  }
  Cache(int64_t hkv_, int64_t dq_) : nb(0), hkv(hkv_), dq(dq_), dv(64), k(nullptr), v(nullptr) {}  // none
};

template <typename T>
T* array_i32(PyObject* o, long dev, int64_t n, const char* what) {
  const int64_t shape[1] = {n};
  return static_cast<T*>(array(o, at::kInt, dev, shape, what));
}

const float* scale(PyObject* o, long dev, int64_t hkv, const char* what) {
  const int64_t shape[1] = {hkv};
  return static_cast<const float*>(array(o, at::kFloat, dev, shape, what));
}

const int32_t* table(PyObject* o, long dev, int64_t batch, int64_t* width) {
  *width = of_dims(o, 2, "block_table").size(1);
  const int64_t shape[2] = {batch, *width};
  return static_cast<const int32_t*>(array(o, at::kInt, dev, shape, "block_table"));
}

// Whole numbers that the library takes in 32 bits.
template <int N>
void check_32(const int64_t (&v)[N]) {
  for (int i = 0; i < N; ++i)
    if (v[i] < INT32_MIN || v[i] > INT32_MAX) refuse("a size does not fit 32 bits");
}

// Runs a call; its status as a Python number, or the error it raised.
template <typename F>
PyObject* entry(Py_ssize_t n, Py_ssize_t want, F call) {
  if (n != want) return PyErr_Format(PyExc_TypeError, "expected %zd arguments, not %zd", want, n);
  try {
    return PyLong_FromLong(call());
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

struct NoGil {
  PyThreadState* state = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(state); }
};

// rope(dev, stream, q, k, v, cos_sin, k_cache, v_cache, k_scale, v_scale,
//      block_table, cu_seqlens_q, ctx_lens, q_out, k_out, rot_start, interleaved)
PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 17, [&]() -> int {
    const long dev = PyLong_AsLong(a[0]);
    void* stream = PyLong_AsVoidPtr(a[1]);
    const long rot_start = PyLong_AsLong(a[15]);
    const int il = PyObject_IsTrue(a[16]);
    check_python();
    const bool fp8 = a[8] != Py_None;
    const at::Tensor& tk = of_dims(a[3], 3, "k");
    const int64_t T = tk.size(0), hkv = tk.size(1), dq = tk.size(2);
    const Rows k(a[3], dev, T, hkv, dq, "k");
    const int64_t batch = of_dims(a[11], 1, "cu_seqlens_q").size(0) - 1;
    const int32_t* cu = array_i32<const int32_t>(a[11], dev, batch + 1, "cu_seqlens_q");
    const int32_t* ctx = a[12] != Py_None ? array_i32<const int32_t>(a[12], dev, batch, "ctx_lens") : nullptr;
    Cache c(hkv, dq);
    Rows v, q, qo, ko;
    const int32_t* bt = nullptr;
    int64_t heads = 0, width = 0, rows = 0, rot = 0;
    if (a[6] != Py_None) {
      c = Cache(a[6], a[7], fp8, dev);
      if (c.hkv != hkv || c.dq != dq) refuse("k and the key cache have different heads or head dims");
      bt = table(a[10], dev, batch, &width);
      v = Rows(a[4], dev, T, hkv, c.dv, "v");
    }
    const float* ks = fp8 ? scale(a[8], dev, hkv, "k_scale") : nullptr;
    const float* vs = fp8 ? scale(a[9], dev, hkv, "v_scale") : nullptr;
    if (a[2] != Py_None) {
      heads = of_dims(a[2], 3, "q").size(1);
      q = Rows(a[2], dev, T, heads, dq, "q");
      qo = Rows(a[13], dev, T, heads, dq, "q_out");
    } else if (a[13] != Py_None) {
      refuse("q_out without q");
    }
    if (a[14] != Py_None) ko = Rows(a[14], dev, T, hkv, dq, "k_out");
    const float* cs = nullptr;
    if (a[5] != Py_None) {
      const at::Tensor& t = of_dims(a[5], 2, "cos_sin");
      rows = t.size(0);
      rot = t.size(1);
      const int64_t shape[2] = {rows, rot};
      cs = static_cast<const float*>(array(a[5], at::kFloat, dev, shape, "cos_sin"));
    }
    check_32({rows, rot_start, rot, width, c.nb, batch, heads, hkv, dq, c.dv});
    const int32_t R = static_cast<int32_t>(rows), W = static_cast<int32_t>(width), NB = static_cast<int32_t>(c.nb),
                  B = static_cast<int32_t>(batch);
    const int s0 = static_cast<int>(rot_start), r = static_cast<int>(rot), H = static_cast<int>(heads),
              G = static_cast<int>(hkv), D = static_cast<int>(dq), E = static_cast<int>(c.dv);
    const NoGil no_gil;
    return fp8 ? f_rope_fp8(q.p, q.stride, k.p, k.stride, v.p, v.stride, cs, R, s0, r, il, qo.p, qo.stride, ko.p, ko.stride,
                            c.k, c.v, ks, vs, bt, W, NB, cu, ctx, B, T, H, G, D, E, stream)
               : f_rope(q.p, q.stride, k.p, k.stride, v.p, v.stride, cs, R, s0, r, il, qo.p, qo.stride, ko.p, ko.stride, c.k,
                        c.v, bt, W, NB, cu, ctx, B, T, H, G, D, E, stream);
  });
}

// decode(dev, stream, q, k_cache, v_cache, k_scale, v_scale, block_table, ctx_lens,
//        out, lse, softmax_scale, workspace address, workspace bytes)
PyObject* py_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 14, [&]() -> int {
    const long dev = PyLong_AsLong(a[0]);
    void* stream = PyLong_AsVoidPtr(a[1]);
    const float softmax_scale = static_cast<float>(PyFloat_AsDouble(a[11]));
    void* ws = PyLong_AsVoidPtr(a[12]);
    const size_t ws_bytes = PyLong_AsSize_t(a[13]);
    check_python();
    const bool fp8 = a[5] != Py_None;
    const at::Tensor& tq = of_dims(a[2], 3, "q");
    const int64_t batch = tq.size(0), heads = tq.size(1);
    const Cache c(a[3], a[4], fp8, dev);
    const Rows q(a[2], dev, batch, heads, c.dq, "q");
    int64_t width;
    const int32_t* bt = table(a[7], dev, batch, &width);
    const int32_t* ctx = array_i32<const int32_t>(a[8], dev, batch, "ctx_lens");
    const float* ks = fp8 ? scale(a[5], dev, c.hkv, "k_scale") : nullptr;
    const float* vs = fp8 ? scale(a[6], dev, c.hkv, "v_scale") : nullptr;
    const int64_t os[3] = {batch, heads, c.dv}, ls[2] = {heads, batch};
    void* out = array(a[9], at::kBFloat16, dev, os, "out");
    float* lse = a[10] != Py_None ? static_cast<float*>(array(a[10], at::kFloat, dev, ls, "lse")) : nullptr;
    check_32({width, c.nb, batch, heads, c.hkv, c.dq, c.dv});
    const int32_t W = static_cast<int32_t>(width), NB = static_cast<int32_t>(c.nb), B = static_cast<int32_t>(batch);
    const int H = static_cast<int>(heads), G = static_cast<int>(c.hkv), D = static_cast<int>(c.dq), E = static_cast<int>(c.dv);
    const NoGil no_gil;
    return fp8 ? f_decode_fp8(q.p, q.stride, c.k, c.v, ks, vs, bt, W, NB, ctx, B, H, G, D, E, softmax_scale, out, lse, ws,
                              ws_bytes, stream)
               : f_decode(q.p, q.stride, c.k, c.v, bt, W, NB, ctx, B, H, G, D, E, softmax_scale, out, lse, ws, ws_bytes, stream);
  });
}

// prompt(dev, stream, q, k, v, cu_seqlens, out, lse, softmax_scale)
PyObject* py_prompt(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 9, [&]() -> int {
    const long dev = PyLong_AsLong(a[0]);
    void* stream = PyLong_AsVoidPtr(a[1]);
    const float softmax_scale = static_cast<float>(PyFloat_AsDouble(a[8]));
    check_python();
    const at::Tensor &tq = of_dims(a[2], 3, "q"), &tv = of_dims(a[4], 3, "v");
    const int64_t T = tq.size(0), heads = tq.size(1), dq = tq.size(2), hkv = tv.size(1), dv = tv.size(2);
    const Rows q(a[2], dev, T, heads, dq, "q"), k(a[3], dev, T, hkv, dq, "k"), v(a[4], dev, T, hkv, dv, "v");
    const int64_t batch = of_dims(a[5], 1, "cu_seqlens").size(0) - 1;
    const int32_t* cu = array_i32<const int32_t>(a[5], dev, batch + 1, "cu_seqlens");
    const int64_t os[3] = {T, heads, dv}, ls[2] = {heads, T};
    void* out = array(a[6], at::kBFloat16, dev, os, "out");
    float* lse = a[7] != Py_None ? static_cast<float*>(array(a[7], at::kFloat, dev, ls, "lse")) : nullptr;
    check_32({batch, heads, hkv, dq, dv});
    const NoGil no_gil;
    return f_prompt(q.p, q.stride, k.p, k.stride, v.p, v.stride, cu, static_cast<int32_t>(batch), T, static_cast<int>(heads),
                    static_cast<int>(hkv), static_cast<int>(dq), static_cast<int>(dv), softmax_scale, out, lse, stream);
  });
}

// setup(addresses of the five functions)
PyObject* py_setup(PyObject*, PyObject* args) {
  PyObject* a[5];
  if (!PyArg_ParseTuple(args, "(OOOOO)", &a[0], &a[1], &a[2], &a[3], &a[4])) return nullptr;
  void* f[5];
  for (int i = 0; i < 5; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (!f[i]) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "a function's address is NULL");
  }
  f_rope = reinterpret_cast<decltype(f_rope)>(f[0]);
  f_rope_fp8 = reinterpret_cast<decltype(f_rope_fp8)>(f[1]);
  f_decode = reinterpret_cast<decltype(f_decode)>(f[2]);
  f_decode_fp8 = reinterpret_cast<decltype(f_decode_fp8)>(f[3]);
  f_prompt = reinterpret_cast<decltype(f_prompt)>(f[4]);
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"setup", py_setup, METH_VARARGS, "Function addresses; called once before the others."},
    {"rope", fast(py_rope), METH_FASTCALL, "vpp_rope_append / _fp8; returns its status."},
    {"decode", fast(py_decode), METH_FASTCALL, "vpp_decode_attn / _fp8; returns its status."},
    {"prompt", fast(py_prompt), METH_FASTCALL, "vpp_prompt_attn; returns its status."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_vppcall", "Calls of the serving-step operators.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__vppcall() { return PyModule_Create(&module); }
