/*
 * marshal_attend.c -- Python calls of the rotary positions with several axes, of scored and of shared attention, straight
 * to the C ABI, for the reason and in the manner of marshal.c: the common case of a call is checked and passed on here
 * (a step's rotation takes 2 us on the GPU and 16 us from Python code); None, with nothing launched, leaves it to the
 * binding's Python code.
 */
#include "marshal.h"

static PyObject *g_f32;

/* rope_axes(q, k | None, positions, pair_axis, inv_freq, magnitude, interleaved, out_q | None, out_k | None)
 *     -> (out_q, out_k) */
static PyObject *rope_axes(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 9) Py_RETURN_NONE;
    PyObject *dtype;
    long long dev, nq[4], nk[4] = {0, 0, 0, 0}, no[4], np[4], qs, ks = 0, oqs, oks = 0;
    const int dt = operand(a[0], &dtype, &dev);
    const int has_k = a[1] != Py_None;
    if (dt < 0 || (!has_k && a[8] != Py_None)) Py_RETURN_NONE;
    int ok = 1;
    void *q = want_rows(a[0], dtype, dev, nq, &qs, &ok), *k = NULL;
    if (has_k) k = want_rows(a[1], dtype, dev, nk, &ks, &ok);
    if (!ok || (has_k && (nk[0] != nq[0] || nk[2] != nq[2] || nk[1] == 0)) || (PyObject *)Py_TYPE(a[2]) != g_tensor)
        Py_RETURN_NONE;
    const int wide = is_dtype(a[2], g_i64);
    void *pos = want(a[2], wide ? g_i64 : g_i32, dev, &ok);
    int32_t *axis = (int32_t *)want(a[3], g_i32, dev, &ok);
    double *freq = (double *)want(a[4], g_f64, dev, &ok);
    if (!ok || sizes(a[2], np) != 2 || np[0] == 0 || np[1] != nq[0]) Py_RETURN_NONE;
    const long long pairs = count(a[4]);
    const double magnitude = PyFloat_AsDouble(a[5]);
    const int interleaved = PyObject_IsTrue(a[6]);
    if (PyErr_Occurred() || interleaved < 0 || pairs < 0 || pairs > 0x3fffffffLL || count(a[3]) != pairs) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    void *stream;
    if (!raw_stream(dev, &stream)) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    PyObject *oq = a[7] == Py_None ? PyObject_CallOneArg(g_empty_like, a[0]) : Py_NewRef(a[7]);
    PyObject *ok_ = !oq ? NULL : !has_k ? Py_NewRef(Py_None) : a[8] == Py_None ? PyObject_CallOneArg(g_empty_like, a[1]) : Py_NewRef(a[8]);
    if (!oq || !ok_) {
        Py_XDECREF(oq);
        return NULL;
    }
    /* (a copy like tokens without gaps needs no look) */
    void *to_q, *to_k = NULL;
    if (a[7] == Py_None && qs == nq[1] * nq[2]) {
        to_q = address(oq, &ok);
        oqs = qs;
    } else {
        to_q = want_rows(oq, dtype, dev, no, &oqs, &ok);
        for (int i = 0; ok && i < 3; ++i) ok = no[i] == nq[i];
    }
    if (has_k && a[8] == Py_None && ks == nk[1] * nk[2]) {
        to_k = address(ok_, &ok);
        oks = ks;
    } else if (has_k) {
        to_k = want_rows(ok_, dtype, dev, no, &oks, &ok);
        for (int i = 0; ok && i < 3; ++i) ok = no[i] == nk[i];
    }
    int rc = PA_ERR_INVALID_ARG;
    if (ok) {
        Py_BEGIN_ALLOW_THREADS;
        rc = pa_rope_axes(to_q, to_k, q, k, oqs, oks, qs, ks, pos, wide ? 8 : 4, np[1], (int)np[0], axis, freq,
                          (float)magnitude, (int)nq[0], (int)nq[1], (int)nk[1], (int)nq[2], (int)(2 * pairs), interleaved,
                          dt, stream);
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

/* A tensor of `dtype` with n entries, or None (NULL). */
static void *maybe(PyObject *t, PyObject *dtype, long long dev, long long n, int *ok) {
    if (t == Py_None || !*ok) return NULL;
    void *p = want(t, dtype, dev, ok);
    if (*ok && count(t) != n) *ok = 0;
    return p;
}

/* attend(q, k_cache, v_cache, block_tables, context_lens, query_start | None, scale, num_kv_heads, max_q, out | None,
 *        cap, slopes | None, first_key | None, bidirectional | None)    or, of 13,
 *        .., prefix_tables, prefix_lens, group_start) -> out */
static PyObject *attend(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 13 && nargs != 14) Py_RETURN_NONE;
    const int shared = nargs == 13;
    PyObject *dtype;
    long long dev, nq[4], nc[4], nv[4], no[4], np[4] = {0, 0, 0, 0};
    const int dt = operand(a[0], &dtype, &dev);
    if (dt < 0) Py_RETURN_NONE;
    tables_t t;
    int ok = 1;
    void *q = want(a[0], dtype, dev, &ok), *kc = want(a[1], dtype, dev, &ok), *vc = want(a[2], dtype, dev, &ok);
    if (!ok || sizes(a[0], nq) != 3 || sizes(a[1], nc) != 4 || sizes(a[2], nv) != 4 ||
        !want_tables(a[3], a[4], a[5], dev, &t))
        Py_RETURN_NONE;
    for (int i = 0; i < 4; ++i)
        if (nc[i] != nv[i]) Py_RETURN_NONE;
    const double scale = PyFloat_AsDouble(a[6]);
    double cap = shared ? 0.0 : PyFloat_AsDouble(a[10]);
    const long long hkv = PyLong_AsLongLong(a[7]), max_q = PyLong_AsLongLong(a[8]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    if (hkv != nc[1] || nq[2] != nc[3] || (!t.qs && nq[0] != t.S) || max_q < 1 || max_q > 0x7fffffffLL) Py_RETURN_NONE;
    if (cap > 0.0 && cap < 0x1p-126) cap = 0x1p-126; /* (fp32 would have none) */
    float *slopes = NULL;
    int32_t *first = NULL, *bidirectional = NULL, *pt = NULL, *pl = NULL, *gs = NULL;
    if (shared) {
        pt = (int32_t *)want(a[10], g_i32, dev, &ok);
        if (!ok || sizes(a[10], np) != 2 || a[11] == Py_None || a[12] == Py_None) Py_RETURN_NONE;
        pl = (int32_t *)maybe(a[11], g_i32, dev, np[0], &ok);
        gs = (int32_t *)maybe(a[12], g_i32, dev, np[0] + 1, &ok);
    } else {
        slopes = (float *)maybe(a[11], g_f32, dev, nq[1], &ok);
        first = (int32_t *)maybe(a[12], g_i32, dev, nq[0], &ok);
        bidirectional = (int32_t *)maybe(a[13], g_i32, dev, t.S, &ok);
    }
    void *stream;
    if (!ok || !raw_stream(dev, &stream)) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    const size_t need = pa_attend_workspace_size((int)t.S, (int)nq[0], (int)max_q, (int)nq[1], (int)hkv, (int)nq[2],
                                                 (int)nc[2], (int)t.max_blocks, (int)np[0], (int)np[1]);
    PyObject *ws = NULL, *out;
    if (need) {
        ws = PyObject_CallFunction(g_workspace, "LKOK", dev, (unsigned long long)(uintptr_t)stream, Py_None,
                                   (unsigned long long)need);
        if (!ws) return NULL;
    }
    out = a[9] == Py_None ? PyObject_CallOneArg(g_empty_like, a[0]) : Py_NewRef(a[9]);
    if (!out) {
        Py_XDECREF(ws);
        return NULL;
    }
    void *o;
    if (a[9] == Py_None) { /* like q, which is contiguous */
        o = address(out, &ok);
    } else {
        o = want(out, dtype, dev, &ok);
        if (ok) ok = sizes(out, no) == 3 && no[0] == nq[0] && no[1] == nq[1] && no[2] == nq[2];
    }
    void *w = ws ? address(ws, &ok) : NULL;
    int rc = PA_ERR_INVALID_ARG;
    if (ok) {
        const int S = (int)t.S, T = (int)nq[0], mq = (int)max_q, hq = (int)nq[1], D = (int)nq[2], B = (int)nc[2],
                  nb = (int)nc[0], mb = (int)t.max_blocks, h = (int)hkv;
        Py_BEGIN_ALLOW_THREADS;
        if (shared && t.qs)
            rc = pa_multi_query_shared(o, q, kc, vc, t.bt, t.cl, t.qs, pt, pl, gs, (int)np[0], (int)np[1], (float)scale, h,
                                       S, T, mq, hq, D, B, nb, mb, dt, w, need, stream);
        else if (shared)
            rc = pa_decode_shared(o, q, kc, vc, t.bt, t.cl, pt, pl, gs, (int)np[0], (int)np[1], (float)scale, h, S, hq, D,
                                  B, nb, mb, dt, w, need, stream);
        else if (t.qs)
            rc = pa_multi_query_scored(o, q, kc, vc, t.bt, t.cl, t.qs, (float)scale, (float)cap, slopes, first,
                                       bidirectional, h, S, T, mq, hq, D, B, nb, mb, dt, w, need, stream);
        else
            rc = pa_decode_scored(o, q, kc, vc, t.bt, t.cl, (float)scale, (float)cap, slopes, first, h, S, hq, D, B, nb,
                                  mb, dt, w, need, stream);
        Py_END_ALLOW_THREADS;
    }
    Py_XDECREF(ws);
    if (rc != PA_OK) {
        Py_DECREF(out);
        Py_RETURN_NONE;
    }
    return out;
}

/* setup(torch.Tensor, (float16, bfloat16, int32, int64, float64, float32), torch.empty_like, raw stream of a device,
 *       current device, workspace(dev, raw stream, None, bytes)) */
static PyObject *setup(PyObject *self, PyObject *args) {
    (void)self;
    PyObject *t, *d[6], *e, *r, *g, *w;
    if (!PyArg_ParseTuple(args, "O(OOOOOO)OOOO", &t, &d[0], &d[1], &d[2], &d[3], &d[4], &d[5], &e, &r, &g, &w)) return NULL;
    PyObject **to[] = {&g_tensor, &g_f16, &g_bf16, &g_i32, &g_i64, &g_f64, &g_f32,
                       &g_empty_like, &g_raw_stream, &g_device, &g_workspace};
    PyObject *from[] = {t, d[0], d[1], d[2], d[3], d[4], d[5], e, r, g, w};
    for (int i = 0; i < 11; ++i) Py_XSETREF(*to[i], Py_NewRef(from[i]));
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, NULL},
    {"attend", (PyCFunction)(void (*)(void))attend, METH_FASTCALL, NULL},
    {"rope_axes", (PyCFunction)(void (*)(void))rope_axes, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal_attend", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal_attend(void) { return intern_names() ? NULL : PyModule_Create(&module); }
