/*
 * marshal.c -- Python calls of the rotary positions and the 8-bit cache, straight to the C ABI.
 *
 * Those calls take 2 to 10 us on the GPU; checking eight tensors and passing twenty arguments from
 * Python code takes longer than that (append of one row per sequence: 10 us, of which 3 are the
 * launch).  These functions make the same checks as the binding's Python code for its common case:
 * plain torch.Tensor operands on the current device, the current stream, the workspace left to the
 * binding.  They return None, having launched nothing, whenever anything is not as that case wants it,
 * and whenever the library refuses: the Python code then takes the call, and works out what is wrong.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/pa.h"

static PyObject *g_tensor, *g_f16, *g_bf16, *g_e4m3, *g_i8, *g_i32, *g_i64, *g_f64;
static PyObject *g_empty_like, *g_raw_stream, *g_device, *g_workspace;
static PyObject *s_dtype, *s_shape, *s_get_device, *s_contiguous, *s_data_ptr, *s_stride;

/* One value of a method without arguments; -1 with no Python error left behind. */
static long long ask(PyObject *t, PyObject *method) {
    PyObject *r = PyObject_CallMethodNoArgs(t, method);
    if (!r) {
        PyErr_Clear();
        return -1;
    }
    const long long v = PyLong_AsLongLong(r);
    Py_DECREF(r);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        return -1;
    }
    return v;
}

/* The address of a tensor's data; 0 in *ok when it has none to give (a batched tensor inside torch.vmap is a plain
 * torch.Tensor with a type, a device and a shape, but raises here). */
static void *address(PyObject *t, int *ok) {
    PyObject *r = PyObject_CallMethodNoArgs(t, s_data_ptr);
    const unsigned long long v = r ? PyLong_AsUnsignedLongLong(r) : 0;
    Py_XDECREF(r);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        *ok = 0;
        return NULL;
    }
    return (void *)(uintptr_t)v;
}

static int is_dtype(PyObject *t, PyObject *dtype) {
    PyObject *d = PyObject_GetAttr(t, s_dtype);
    if (!d) {
        PyErr_Clear();
        return 0;
    }
    Py_DECREF(d); /* types are singletons that torch keeps */
    return d == dtype;
}

/* Address of a plain contiguous tensor of `dtype` on device `dev`; 0 in *ok when it is not one. */
static void *want(PyObject *t, PyObject *dtype, long long dev, int *ok) {
    if (!*ok || (PyObject *)Py_TYPE(t) != g_tensor || !is_dtype(t, dtype) || ask(t, s_get_device) != dev ||
        ask(t, s_contiguous) != 1) {
        *ok = 0;
        return NULL;
    }
    return address(t, ok);
}

/* Up to four sizes; the number of dimensions, or -1. */
static int sizes(PyObject *t, long long *n) {
    PyObject *s = PyObject_GetAttr(t, s_shape);
    if (!s) {
        PyErr_Clear();
        return -1;
    }
    int dims = PyTuple_Check(s) ? (int)PyTuple_GET_SIZE(s) : -1;
    if (dims > 4) dims = -1;
    for (int i = 0; i < dims; ++i) {
        n[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(s, i));
        if (n[i] < 0 || n[i] > 0x7fffffffLL) dims = -1;
    }
    Py_DECREF(s);
    PyErr_Clear();
    return dims;
}

/* [T, heads, D] with a token's heads contiguous: address and elements between tokens. */
static void *want_rows(PyObject *t, PyObject *dtype, long long dev, long long *n, long long *stride, int *ok) {
    if (!*ok || (PyObject *)Py_TYPE(t) != g_tensor || !is_dtype(t, dtype) || ask(t, s_get_device) != dev ||
        sizes(t, n) != 3) {
        *ok = 0;
        return NULL;
    }
    *stride = n[1] * n[2];
    if (ask(t, s_contiguous) != 1) {
        PyObject *st = PyObject_CallMethodNoArgs(t, s_stride);
        if (!st || !PyTuple_Check(st) || PyTuple_GET_SIZE(st) != 3) {
            PyErr_Clear();
            Py_XDECREF(st);
            *ok = 0;
            return NULL;
        }
        const long long a = PyLong_AsLongLong(PyTuple_GET_ITEM(st, 0)), b = PyLong_AsLongLong(PyTuple_GET_ITEM(st, 1)),
                        c = PyLong_AsLongLong(PyTuple_GET_ITEM(st, 2));
        Py_DECREF(st);
        PyErr_Clear();
        if (c != 1 || (n[1] > 1 && b != n[2])) {
            *ok = 0;
            return NULL;
        }
        if (n[0] > 1) *stride = a;
    }
    return address(t, ok);
}

/* The 16-bit type of `t` and its library number (-1: none), and its device if that is the current one. */
static int operand(PyObject *t, PyObject **dtype, long long *dev) {
    if ((PyObject *)Py_TYPE(t) != g_tensor) return -1;
    *dev = ask(t, s_get_device);
    if (*dev < 0) return -1;
    PyObject *d = PyObject_CallNoArgs(g_device);
    if (!d) {
        PyErr_Clear();
        return -1;
    }
    const long long now = PyLong_AsLongLong(d);
    Py_DECREF(d);
    if (now != *dev) return -1;
    if (is_dtype(t, g_f16)) {
        *dtype = g_f16;
        return PA_F16;
    }
    if (is_dtype(t, g_bf16)) {
        *dtype = g_bf16;
        return PA_BF16;
    }
    return -1;
}

static int raw_stream(long long dev, void **stream) {
    PyObject *d = PyLong_FromLongLong(dev);
    PyObject *r = d ? PyObject_CallOneArg(g_raw_stream, d) : NULL;
    Py_XDECREF(d);
    if (!r) {
        PyErr_Clear();
        return 0;
    }
    *stream = (void *)(uintptr_t)PyLong_AsUnsignedLongLong(r);
    Py_DECREF(r);
    return !PyErr_Occurred();
}

typedef struct {
    void *k, *v;
    int8_t *ke, *ve;
    long long n[4]; /* NB, Hkv, B, D */
} cache_t;

static int want_cache(PyObject *const *a, long long dev, cache_t *c) {
    int ok = 1;
    long long m[4];
    c->k = want(a[0], g_e4m3, dev, &ok);
    c->v = want(a[1], g_e4m3, dev, &ok);
    c->ke = (int8_t *)want(a[2], g_i8, dev, &ok);
    c->ve = (int8_t *)want(a[3], g_i8, dev, &ok);
    if (!ok || sizes(a[0], c->n) != 4 || sizes(a[1], m) != 4) return 0;
    for (int i = 0; i < 4; ++i)
        if (m[i] != c->n[i]) return 0;
    for (int i = 2; i < 4; ++i)
        if (sizes(a[i], m) != 2 || m[0] != c->n[0] || m[1] != c->n[1]) return 0;
    return 1;
}

/* block_tables [S, max_blocks], context_lens (S entries), query_start (S + 1 entries, or None) */
typedef struct {
    int32_t *bt, *cl, *qs;
    long long S, max_blocks;
} tables_t;

static long long count(PyObject *t) {
    long long n[4], c = 1;
    const int dims = sizes(t, n);
    if (dims < 0) return -1;
    for (int i = 0; i < dims; ++i) {
        c *= n[i];
        if (c > 0x7fffffffLL) return -1;
    }
    return c;
}

static int want_tables(PyObject *bt, PyObject *cl, PyObject *qs, long long dev, tables_t *t) {
    int ok = 1;
    long long n[4];
    t->bt = (int32_t *)want(bt, g_i32, dev, &ok);
    t->cl = (int32_t *)want(cl, g_i32, dev, &ok);
    t->qs = qs == Py_None ? NULL : (int32_t *)want(qs, g_i32, dev, &ok);
    if (!ok || sizes(bt, n) != 2) return 0;
    t->S = count(cl);
    t->max_blocks = n[1];
    return n[0] == t->S && (qs == Py_None || count(qs) == t->S + 1);
}

/* attention(q, k_cache, v_cache, k_exp, v_exp, block_tables, context_lens, query_start | None, scale, num_kv_heads,
 *           max_q, out | None) -> out */
static PyObject *attention(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 12) Py_RETURN_NONE;
    PyObject *dtype;
    long long dev, nq[4], no[4];
    const int dt = operand(a[0], &dtype, &dev);
    if (dt < 0) Py_RETURN_NONE;
    cache_t c;
    tables_t t;
    int ok = 1;
    void *q = want(a[0], dtype, dev, &ok);
    if (!ok || sizes(a[0], nq) != 3 || !want_cache(a + 1, dev, &c) || !want_tables(a[5], a[6], a[7], dev, &t))
        Py_RETURN_NONE;
    const double scale = PyFloat_AsDouble(a[8]);
    const long long hkv = PyLong_AsLongLong(a[9]), max_q = PyLong_AsLongLong(a[10]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    if (hkv != c.n[1] || nq[2] != c.n[3] || (!t.qs && nq[0] != t.S) || max_q < 1 || max_q > 0x7fffffffLL) Py_RETURN_NONE;
    void *stream;
    if (!raw_stream(dev, &stream)) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    const size_t need = pa_decode_q8_workspace_size((int)t.S, (int)nq[1], (int)hkv, (int)nq[2], (int)c.n[2],
                                                    (int)t.max_blocks, (int)max_q);
    PyObject *ws = NULL, *out;
    if (need) {
        ws = PyObject_CallFunction(g_workspace, "LKOK", dev, (unsigned long long)(uintptr_t)stream, Py_None,
                                   (unsigned long long)need);
        if (!ws) return NULL;
    }
    if (a[11] == Py_None) {
        out = PyObject_CallOneArg(g_empty_like, a[0]);
        if (!out) {
            Py_XDECREF(ws);
            return NULL;
        }
    } else {
        out = Py_NewRef(a[11]);
    }
    void *o;
    if (a[11] == Py_None) { /* like q, which is contiguous */
        o = address(out, &ok);
    } else {
        o = want(out, dtype, dev, &ok);
        if (ok) ok = sizes(out, no) == 3 && no[0] == nq[0] && no[1] == nq[1] && no[2] == nq[2];
    }
    void *w = ws ? address(ws, &ok) : NULL;
    int rc = PA_ERR_INVALID_ARG;
    if (ok) {
        Py_BEGIN_ALLOW_THREADS;
        if (t.qs)
            rc = pa_multi_query_q8(o, q, c.k, c.v, c.ke, c.ve, t.bt, t.cl, t.qs, (float)scale, (int)hkv, (int)t.S,
                                   (int)nq[0], (int)max_q, (int)nq[1], (int)nq[2], (int)c.n[2], (int)c.n[0],
                                   (int)t.max_blocks, dt, w, need, stream);
        else
            rc = pa_decode_q8(o, q, c.k, c.v, c.ke, c.ve, t.bt, t.cl, (float)scale, (int)hkv, (int)t.S, (int)nq[1],
                              (int)nq[2], (int)c.n[2], (int)c.n[0], (int)t.max_blocks, dt, w, need, stream);
        Py_END_ALLOW_THREADS;
    }
    Py_XDECREF(ws);
    if (rc != PA_OK) {
        Py_DECREF(out);
        Py_RETURN_NONE;
    }
    return out;
}

/* append(k, v, k_cache, v_cache, k_exp, v_exp, block_tables, context_lens, query_start | None, max_q) -> True */
static PyObject *append(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 10) Py_RETURN_NONE;
    PyObject *dtype;
    long long dev, nk[4], nv[4], ks, vs;
    const int dt = operand(a[0], &dtype, &dev);
    if (dt < 0) Py_RETURN_NONE;
    cache_t c;
    tables_t t;
    int ok = 1;
    void *k = want_rows(a[0], dtype, dev, nk, &ks, &ok), *v = want_rows(a[1], dtype, dev, nv, &vs, &ok);
    if (!ok || !want_cache(a + 2, dev, &c) || !want_tables(a[6], a[7], a[8], dev, &t)) Py_RETURN_NONE;
    const long long max_q = t.qs ? PyLong_AsLongLong(a[9]) : 1;
    if (PyErr_Occurred()) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    if (nk[1] != c.n[1] || nk[2] != c.n[3] || nv[0] != nk[0] || nv[1] != nk[1] || nv[2] != nk[2] ||
        (!t.qs && nk[0] != t.S) || max_q < 1 || max_q > 0x7fffffffLL)
        Py_RETURN_NONE;
    void *stream;
    if (!raw_stream(dev, &stream)) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = pa_cache_append_q8(k, v, ks, vs, c.k, c.v, c.ke, c.ve, t.bt, t.cl, t.qs, (int)t.S, (int)nk[0], (int)max_q,
                            (int)c.n[1], (int)c.n[3], (int)c.n[2], (int)c.n[0], (int)t.max_blocks, dt, stream);
    Py_END_ALLOW_THREADS;
    if (rc != PA_OK) Py_RETURN_NONE;
    Py_RETURN_TRUE;
}

/* read_blocks(k_cache, v_cache, k_exp, v_exp, dst_k, dst_v, src_ids, dst_ids) -> True */
static PyObject *read_blocks(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 8) Py_RETURN_NONE;
    PyObject *dtype;
    long long dev, n[4], m[4];
    const int dt = operand(a[4], &dtype, &dev);
    if (dt < 0) Py_RETURN_NONE;
    cache_t c;
    int ok = 1;
    void *dk = want(a[4], dtype, dev, &ok), *dv = want(a[5], dtype, dev, &ok);
    int32_t *src = (int32_t *)want(a[6], g_i32, dev, &ok), *dst = (int32_t *)want(a[7], g_i32, dev, &ok);
    if (!ok || !want_cache(a, dev, &c) || sizes(a[4], n) != 4 || sizes(a[5], m) != 4) Py_RETURN_NONE;
    const long long pairs = count(a[6]);
    if (pairs < 0 || count(a[7]) != pairs || m[0] != n[0]) Py_RETURN_NONE;
    for (int i = 1; i < 4; ++i)
        if (n[i] != c.n[i] || m[i] != n[i]) Py_RETURN_NONE;
    void *stream;
    if (!raw_stream(dev, &stream)) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = pa_read_blocks_q8(c.k, c.v, c.ke, c.ve, (int)c.n[0], dk, dv, (int)n[0], src, dst, (int)pairs, (int)c.n[1],
                           (int)c.n[3], (int)c.n[2], dt, stream);
    Py_END_ALLOW_THREADS;
    if (rc != PA_OK) Py_RETURN_NONE;
    Py_RETURN_TRUE;
}

/* rope(q, k | None, positions, inv_freq, magnitude, interleaved, out_q | None, out_k | None) -> (out_q, out_k) */
static PyObject *rope(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 8) Py_RETURN_NONE;
    PyObject *dtype;
    long long dev, nq[4], nk[4] = {0, 0, 0, 0}, no[4], qs, ks = 0, oqs, oks = 0;
    const int dt = operand(a[0], &dtype, &dev);
    const int has_k = a[1] != Py_None;
    if (dt < 0 || (!has_k && a[7] != Py_None)) Py_RETURN_NONE;
    int ok = 1;
    void *q = want_rows(a[0], dtype, dev, nq, &qs, &ok), *k = NULL;
    if (has_k) k = want_rows(a[1], dtype, dev, nk, &ks, &ok);
    if (!ok || (has_k && (nk[0] != nq[0] || nk[2] != nq[2] || nk[1] == 0)) || (PyObject *)Py_TYPE(a[2]) != g_tensor)
        Py_RETURN_NONE;
    const int wide = is_dtype(a[2], g_i64);
    void *pos = want(a[2], wide ? g_i64 : g_i32, dev, &ok);
    double *freq = (double *)want(a[3], g_f64, dev, &ok);
    if (!ok || count(a[2]) != nq[0]) Py_RETURN_NONE;
    const long long pairs = count(a[3]);
    const double magnitude = PyFloat_AsDouble(a[4]);
    const int interleaved = PyObject_IsTrue(a[5]);
    if (PyErr_Occurred() || interleaved < 0 || pairs < 0 || pairs > 0x3fffffffLL) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    void *stream;
    if (!raw_stream(dev, &stream)) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    /* torch.empty_like keeps the strides of a dense tensor only: a slice's copy is contiguous; that of tokens without
     * gaps needs no look */
    PyObject *oq = a[6] == Py_None ? PyObject_CallOneArg(g_empty_like, a[0]) : Py_NewRef(a[6]);
    PyObject *ok_ = !oq ? NULL : !has_k ? Py_NewRef(Py_None) : a[7] == Py_None ? PyObject_CallOneArg(g_empty_like, a[1]) : Py_NewRef(a[7]);
    if (!oq || !ok_) {
        Py_XDECREF(oq);
        return NULL;
    }
    void *to_q, *to_k = NULL;
    if (a[6] == Py_None && qs == nq[1] * nq[2]) {
        to_q = address(oq, &ok);
        oqs = qs;
    } else {
        to_q = want_rows(oq, dtype, dev, no, &oqs, &ok);
        for (int i = 0; ok && i < 3; ++i) ok = no[i] == nq[i];
    }
    if (has_k && a[7] == Py_None && ks == nk[1] * nk[2]) {
        to_k = address(ok_, &ok);
        oks = ks;
    } else if (has_k) {
        to_k = want_rows(ok_, dtype, dev, no, &oks, &ok);
        for (int i = 0; ok && i < 3; ++i) ok = no[i] == nk[i];
    }
    int rc = PA_ERR_INVALID_ARG;
    if (ok) {
        Py_BEGIN_ALLOW_THREADS;
        rc = pa_rope(to_q, to_k, q, k, oqs, oks, qs, ks, pos, wide ? 8 : 4, freq, (float)magnitude, (int)nq[0], (int)nq[1],
                     (int)nk[1], (int)nq[2], (int)(2 * pairs), interleaved, dt, stream);
        Py_END_ALLOW_THREADS;
    }
    if (rc != PA_OK) {
        Py_DECREF(oq);
        Py_DECREF(ok_);
        Py_RETURN_NONE;
    }
    PyObject *both = PyTuple_Pack(2, oq, ok_);
    Py_DECREF(oq);
    Py_DECREF(ok_);
    return both;
}

/* setup(torch.Tensor, (float16, bfloat16, float8_e4m3fn, int8, int32, int64, float64), torch.empty_like,
 *       raw stream of a device, current device, workspace(dev, raw stream, None, bytes)) */
static PyObject *setup(PyObject *self, PyObject *args) {
    (void)self;
    PyObject *t, *d[7], *e, *r, *g, *w;
    if (!PyArg_ParseTuple(args, "O(OOOOOOO)OOOO", &t, &d[0], &d[1], &d[2], &d[3], &d[4], &d[5], &d[6], &e, &r, &g, &w))
        return NULL;
    PyObject **to[] = {&g_tensor, &g_f16, &g_bf16, &g_e4m3, &g_i8, &g_i32, &g_i64, &g_f64,
                       &g_empty_like, &g_raw_stream, &g_device, &g_workspace};
    PyObject *from[] = {t, d[0], d[1], d[2], d[3], d[4], d[5], d[6], e, r, g, w};
    for (int i = 0; i < 12; ++i) Py_XSETREF(*to[i], Py_NewRef(from[i]));
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, NULL},
    {"attention", (PyCFunction)(void (*)(void))attention, METH_FASTCALL, NULL},
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, NULL},
    {"read_blocks", (PyCFunction)(void (*)(void))read_blocks, METH_FASTCALL, NULL},
    {"rope", (PyCFunction)(void (*)(void))rope, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void) {
    PyObject **names[] = {&s_dtype, &s_shape, &s_get_device, &s_contiguous, &s_data_ptr, &s_stride};
    const char *text[] = {"dtype", "shape", "get_device", "is_contiguous", "data_ptr", "stride"};
    for (int i = 0; i < 6; ++i)
        if (!(*names[i] = PyUnicode_InternFromString(text[i]))) return NULL;
    return PyModule_Create(&module);
}
