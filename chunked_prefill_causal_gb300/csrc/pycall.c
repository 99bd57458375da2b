/*
 * pycall.c -- argument checks and the C calls of the device-planned serving
 * operators, for vpp.py.  Their kernels take a few microseconds at decode sizes,
 * less than ctypes takes to convert thirty arguments; here a tensor's type, shape,
 * strides, device and address are read through Python's C API (no torch headers)
 * and the library's functions are called by address.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>

#include "vpp.h"

static PyObject *s_shape, *s_stride, *s_dtype, *s_get_device, *s_data_ptr, *s_is_contiguous;
static PyObject *t_bf16, *t_f32, *t_i32, *t_u8;

static __typeof__(&vpp_rope_append) f_rope;
static __typeof__(&vpp_rope_append_fp8) f_rope_fp8;
static __typeof__(&vpp_decode_attn) f_decode;
static __typeof__(&vpp_decode_attn_fp8) f_decode_fp8;
static __typeof__(&vpp_prompt_attn) f_prompt;

/* Reads a tuple of whole numbers; returns its length or -1. */
static int sizes(PyObject *tuple, int64_t *out, int most, const char *what) {
    if (!tuple) return -1;
    const Py_ssize_t n = PyTuple_Check(tuple) ? PyTuple_GET_SIZE(tuple) : -1;
    if (n < 0 || n > most) {
        PyErr_Format(PyExc_ValueError, "%s has the wrong number of dimensions", what);
        Py_DECREF(tuple);
        return -1;
    }
    for (Py_ssize_t i = 0; i < n; ++i) {
        out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
        if (out[i] == -1 && PyErr_Occurred()) {
            Py_DECREF(tuple);
            return -1;
        }
    }
    Py_DECREF(tuple);
    return (int)n;
}

static int shape_of(PyObject *t, int64_t *out, int nd, const char *what) {
    const int n = sizes(PyObject_GetAttr(t, s_shape), out, 8, what);
    if (n < 0) return -1;
    if (n != nd) {
        PyErr_Format(PyExc_ValueError, "%s must have %d dimensions, not %d", what, nd, n);
        return -1;
    }
    return 0;
}

/* Type and device of a tensor. */
static int kind(PyObject *t, PyObject *dtype, long dev, const char *what) {
    PyObject *d = PyObject_GetAttr(t, s_dtype);
    if (!d) return -1;
    const int same = d == dtype;
    Py_DECREF(d);
    if (!same) {
        PyErr_Format(PyExc_ValueError, "%s must be %S", what, dtype);
        return -1;
    }
    PyObject *g = PyObject_CallMethodNoArgs(t, s_get_device);
    if (!g) return -1;
    const long at = PyLong_AsLong(g);
    Py_DECREF(g);
    if (at != dev || at < 0) {
        PyErr_Format(PyExc_ValueError, "%s must be on the current CUDA device", what);
        return -1;
    }
    return 0;
}

static int contiguous(PyObject *t) {
    PyObject *c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (!c) return -1;
    const int yes = c == Py_True;
    Py_DECREF(c);
    return yes;
}

static int address(PyObject *t, void **out) {
    PyObject *p = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!p) return -1;
    *out = PyLong_AsVoidPtr(p);
    Py_DECREF(p);
    return *out == NULL && PyErr_Occurred() ? -1 : 0;
}

/* Address of a contiguous tensor of this type and shape. */
static int array(PyObject *t, PyObject *dtype, long dev, int nd, const int64_t *shape, const char *what, void **out) {
    int64_t s[8];
    if (kind(t, dtype, dev, what) || shape_of(t, s, nd, what)) return -1;
    for (int i = 0; i < nd; ++i)
        if (s[i] != shape[i]) {
            PyErr_Format(PyExc_ValueError, "%s has the wrong shape: dimension %d is %lld, not %lld", what, i, (long long)s[i],
                         (long long)shape[i]);
            return -1;
        }
    const int c = contiguous(t);
    if (c < 0) return -1;
    if (!c) {
        PyErr_Format(PyExc_ValueError, "%s must be contiguous", what);
        return -1;
    }
    return address(t, out);
}

/* Address and token stride of a bf16 [n, h, d] tensor whose heads are contiguous
 * within a token (a part of a wider projection is).  The stride of a single token
 * is never used and reported as the row's length. */
static int tokens(PyObject *t, long dev, int64_t n, int64_t h, int64_t d, const char *what, void **out, int64_t *stride) {
    int64_t s[8], st[8];
    if (kind(t, t_bf16, dev, what) || shape_of(t, s, 3, what)) return -1;
    if (s[0] != n || s[1] != h || s[2] != d) {
        PyErr_Format(PyExc_ValueError, "%s must be [%lld, %lld, %lld], not [%lld, %lld, %lld]", what, (long long)n,
                     (long long)h, (long long)d, (long long)s[0], (long long)s[1], (long long)s[2]);
        return -1;
    }
    const int c = contiguous(t);
    if (c < 0) return -1;
    *stride = h * d;
    if (!c) {
        if (sizes(PyObject_CallMethodNoArgs(t, s_stride), st, 8, what) < 0) return -1;
        if ((st[2] != 1 && d > 1) || (st[1] != d && h > 1)) {
            PyErr_Format(PyExc_ValueError, "%s: a token's heads must be contiguous", what);
            return -1;
        }
        if (n > 1) *stride = st[0];
    }
    return address(t, out);
}

static int is_none(PyObject *o) { return o == Py_None; }

static int argc_is(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return 0;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, not %zd", want, n);
    return -1;
}

/* A paged cache: blocks, kv heads, dims and addresses. */
typedef struct {
    int64_t nb, hkv, dq, dv;
    void *k, *v;
} Cache;

static int cache(PyObject *k, PyObject *v, PyObject *dtype, long dev, Cache *c) {
    int64_t s[8];
    if (shape_of(k, s, 4, "k_cache")) return -1;
    c->nb = s[0];
    c->hkv = s[2];
    c->dq = s[3];
    if (shape_of(v, s, 4, "v_cache")) return -1;
    c->dv = s[3];
    const int64_t ks[4] = {c->nb, 64, c->hkv, c->dq}, vs[4] = {c->nb, 64, c->hkv, c->dv};
    return array(k, dtype, dev, 4, ks, "k_cache", &c->k) || array(v, dtype, dev, 4, vs, "v_cache", &c->v) ? -1 : 0;
}

static int scales(PyObject *ks, PyObject *vs, long dev, int64_t hkv, void **k, void **v) {
    return array(ks, t_f32, dev, 1, &hkv, "k_scale", k) || array(vs, t_f32, dev, 1, &hkv, "v_scale", v) ? -1 : 0;
}

/* The block table's row length and address. */
static int table(PyObject *t, long dev, int64_t batch, int64_t *width, void **out) {
    int64_t s[8];
    if (shape_of(t, s, 2, "block_table")) return -1;
    *width = s[1];
    const int64_t want[2] = {batch, s[1]};
    return array(t, t_i32, dev, 2, want, "block_table", out);
}

/* Whole numbers that the library takes in 32 bits. */
static int fits(const int64_t *v, int n) {
    for (int i = 0; i < n; ++i)
        if (v[i] < INT32_MIN || v[i] > INT32_MAX) {
            PyErr_SetString(PyExc_ValueError, "a size does not fit 32 bits");
            return -1;
        }
    return 0;
}

/* rope(dev, stream, q, k, v, cos_sin, k_cache, v_cache, k_scale, v_scale,
 *      block_table, cu_seqlens_q, ctx_lens, q_out, k_out, rot_start, interleaved) */
static PyObject *py_rope(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (argc_is(n, 17)) return NULL;
    const long dev = PyLong_AsLong(a[0]);
    void *stream = PyLong_AsVoidPtr(a[1]);
    const long rot_start = PyLong_AsLong(a[15]);
    const int il = PyObject_IsTrue(a[16]);
    if (PyErr_Occurred()) return NULL;
    const int fp8 = !is_none(a[8]);
    void *q = NULL, *k, *v = NULL, *cs = NULL, *bt = NULL, *cu, *ctx = NULL, *qo = NULL, *ko = NULL, *ksc = NULL, *vsc = NULL;
    int64_t qst = 0, kst, vst = 0, qost = 0, kost = 0, s[8], heads = 0, width = 0, rows = 0, rot = 0;
    if (shape_of(a[3], s, 3, "k")) return NULL;
    const int64_t T = s[0], hkv = s[1], dq = s[2];
    if (tokens(a[3], dev, T, hkv, dq, "k", &k, &kst)) return NULL;
    if (shape_of(a[11], s, 1, "cu_seqlens_q")) return NULL;
    const int64_t batch = s[0] - 1;
    if (array(a[11], t_i32, dev, 1, s, "cu_seqlens_q", &cu)) return NULL;
    if (!is_none(a[12]) && array(a[12], t_i32, dev, 1, &batch, "ctx_lens", &ctx)) return NULL;
    Cache c = {0, hkv, dq, 64, NULL, NULL}; /* (no values without a cache) */
    if (!is_none(a[6])) {
        if (cache(a[6], a[7], fp8 ? t_u8 : t_bf16, dev, &c)) return NULL;
        if (c.hkv != hkv || c.dq != dq) {
            PyErr_SetString(PyExc_ValueError, "k and the key cache have different heads or head dims");
            return NULL;
        }
        if (table(a[10], dev, batch, &width, &bt) || tokens(a[4], dev, T, hkv, c.dv, "v", &v, &vst)) return NULL;
    }
    if (fp8 && scales(a[8], a[9], dev, hkv, &ksc, &vsc)) return NULL;
    if (!is_none(a[2])) {
        if (shape_of(a[2], s, 3, "q")) return NULL;
        heads = s[1];
        if (tokens(a[2], dev, T, heads, dq, "q", &q, &qst) || tokens(a[13], dev, T, heads, dq, "q_out", &qo, &qost)) return NULL;
    } else if (!is_none(a[13])) {
        PyErr_SetString(PyExc_ValueError, "q_out without q");
        return NULL;
    }
    if (!is_none(a[14]) && tokens(a[14], dev, T, hkv, dq, "k_out", &ko, &kost)) return NULL;
    if (!is_none(a[5])) {
        if (shape_of(a[5], s, 2, "cos_sin")) return NULL;
        rows = s[0];
        rot = s[1];
        if (array(a[5], t_f32, dev, 2, s, "cos_sin", &cs)) return NULL;
    }
    const int64_t small[] = {rows, rot_start, rot, width, c.nb, batch, heads, hkv, dq, c.dv};
    if (fits(small, 10)) return NULL;
    int code;
    Py_BEGIN_ALLOW_THREADS;
    if (fp8)
        code = f_rope_fp8(q, qst, k, kst, v, vst, cs, (int32_t)rows, (int)rot_start, (int)rot, il, qo, qost, ko, kost, c.k, c.v, ksc,
                          vsc, bt, (int32_t)width, (int32_t)c.nb, cu, ctx, (int32_t)batch, T, (int)heads, (int)hkv, (int)dq,
                          (int)c.dv, stream);
    else
        code = f_rope(q, qst, k, kst, v, vst, cs, (int32_t)rows, (int)rot_start, (int)rot, il, qo, qost, ko, kost, c.k, c.v, bt,
                      (int32_t)width, (int32_t)c.nb, cu, ctx, (int32_t)batch, T, (int)heads, (int)hkv, (int)dq, (int)c.dv, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(code);
}

/* decode(dev, stream, q, k_cache, v_cache, k_scale, v_scale, block_table, ctx_lens,
 *        out, lse, softmax_scale, workspace address, workspace bytes) */
static PyObject *py_decode(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (argc_is(n, 14)) return NULL;
    const long dev = PyLong_AsLong(a[0]);
    void *stream = PyLong_AsVoidPtr(a[1]);
    const double scale = PyFloat_AsDouble(a[11]);
    void *ws = PyLong_AsVoidPtr(a[12]);
    const size_t ws_bytes = PyLong_AsSize_t(a[13]);
    if (PyErr_Occurred()) return NULL;
    const int fp8 = !is_none(a[5]);
    void *q, *bt, *ctx, *out, *lse = NULL, *ksc = NULL, *vsc = NULL;
    int64_t qst, s[8], width;
    if (shape_of(a[2], s, 3, "q")) return NULL;
    const int64_t B = s[0], H = s[1];
    Cache c;
    if (cache(a[3], a[4], fp8 ? t_u8 : t_bf16, dev, &c) || tokens(a[2], dev, B, H, c.dq, "q", &q, &qst) ||
        table(a[7], dev, B, &width, &bt) || array(a[8], t_i32, dev, 1, &B, "ctx_lens", &ctx))
        return NULL;
    if (fp8 && scales(a[5], a[6], dev, c.hkv, &ksc, &vsc)) return NULL;
    const int64_t os[3] = {B, H, c.dv}, ls[2] = {H, B};
    if (array(a[9], t_bf16, dev, 3, os, "out", &out)) return NULL;
    if (!is_none(a[10]) && array(a[10], t_f32, dev, 2, ls, "lse", &lse)) return NULL;
    const int64_t small[] = {width, c.nb, B, H, c.hkv, c.dq, c.dv};
    if (fits(small, 7)) return NULL;
    int code;
    Py_BEGIN_ALLOW_THREADS;
    if (fp8)
        code = f_decode_fp8(q, qst, c.k, c.v, ksc, vsc, bt, (int32_t)width, (int32_t)c.nb, ctx, (int32_t)B, (int)H, (int)c.hkv,
                            (int)c.dq, (int)c.dv, (float)scale, out, lse, ws, ws_bytes, stream);
    else
        code = f_decode(q, qst, c.k, c.v, bt, (int32_t)width, (int32_t)c.nb, ctx, (int32_t)B, (int)H, (int)c.hkv, (int)c.dq,
                        (int)c.dv, (float)scale, out, lse, ws, ws_bytes, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(code);
}

/* prompt(dev, stream, q, k, v, cu_seqlens, out, lse, softmax_scale) */
static PyObject *py_prompt(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (argc_is(n, 9)) return NULL;
    const long dev = PyLong_AsLong(a[0]);
    void *stream = PyLong_AsVoidPtr(a[1]);
    const double scale = PyFloat_AsDouble(a[8]);
    if (PyErr_Occurred()) return NULL;
    void *q, *k, *v, *cu, *out, *lse = NULL;
    int64_t qst, kst, vst, s[8];
    if (shape_of(a[2], s, 3, "q")) return NULL;
    const int64_t T = s[0], H = s[1], dq = s[2];
    if (shape_of(a[4], s, 3, "v")) return NULL;
    const int64_t hkv = s[1], dv = s[2];
    if (tokens(a[2], dev, T, H, dq, "q", &q, &qst) || tokens(a[3], dev, T, hkv, dq, "k", &k, &kst) ||
        tokens(a[4], dev, T, hkv, dv, "v", &v, &vst) || shape_of(a[5], s, 1, "cu_seqlens"))
        return NULL;
    const int64_t batch = s[0] - 1;
    const int64_t os[3] = {T, H, dv}, ls[2] = {H, T};
    if (array(a[5], t_i32, dev, 1, s, "cu_seqlens", &cu) || array(a[6], t_bf16, dev, 3, os, "out", &out)) return NULL;
    if (!is_none(a[7]) && array(a[7], t_f32, dev, 2, ls, "lse", &lse)) return NULL;
    const int64_t small[] = {batch, H, hkv, dq, dv};
    if (fits(small, 5)) return NULL;
    int code;
    Py_BEGIN_ALLOW_THREADS;
    code = f_prompt(q, qst, k, kst, v, vst, cu, (int32_t)batch, T, (int)H, (int)hkv, (int)dq, (int)dv, (float)scale, out, lse, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(code);
}

/* setup((bfloat16, float32, int32, uint8), (addresses of the five functions)) */
static PyObject *py_setup(PyObject *self, PyObject *args) {
    (void)self;
    PyObject *a[9];
    if (!PyArg_ParseTuple(args, "(OOOO)(OOOOO)", &a[0], &a[1], &a[2], &a[3], &a[4], &a[5], &a[6], &a[7], &a[8])) return NULL;
    void *f[5];
    for (int i = 0; i < 5; ++i) {
        f[i] = PyLong_AsVoidPtr(a[4 + i]);
        if (!f[i]) return PyErr_Occurred() ? NULL : PyErr_Format(PyExc_ValueError, "a function's address is NULL");
    }
    PyObject **t[4] = {&t_bf16, &t_f32, &t_i32, &t_u8};
    for (int i = 0; i < 4; ++i) Py_XSETREF(*t[i], Py_NewRef(a[i]));
    f_rope = (__typeof__(f_rope))f[0];
    f_rope_fp8 = (__typeof__(f_rope_fp8))f[1];
    f_decode = (__typeof__(f_decode))f[2];
    f_decode_fp8 = (__typeof__(f_decode_fp8))f[3];
    f_prompt = (__typeof__(f_prompt))f[4];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", py_setup, METH_VARARGS, "Types and function addresses; called once before the others."},
    {"rope", (PyCFunction)(void (*)(void))py_rope, METH_FASTCALL, "vpp_rope_append / _fp8; returns its status."},
    {"decode", (PyCFunction)(void (*)(void))py_decode, METH_FASTCALL, "vpp_decode_attn / _fp8; returns its status."},
    {"prompt", (PyCFunction)(void (*)(void))py_prompt, METH_FASTCALL, "vpp_prompt_attn; returns its status."},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_vppcall", "Calls of the serving-step operators.", -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__vppcall(void) {
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    if (!s_shape || !s_stride || !s_dtype || !s_get_device || !s_data_ptr || !s_is_contiguous) return NULL;
    return PyModule_Create(&module);
}
