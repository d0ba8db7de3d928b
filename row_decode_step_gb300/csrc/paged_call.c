/*
 * CPython side of the paged cache's calls: checks the tensors and calls the library.
 *
 * A decode step makes these calls once a layer and they take microseconds on the GPU, so their host
 * time counts: the same checks written in Python and marshalled by ctypes took 4 us more a call.
 * Tensors are read through their public methods (dtype, get_device, shape, stride, data_ptr); no torch
 * header is needed.  row_decode_step_gb300/paged.py holds the calls a user makes.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "dl.h"

typedef int (*append_fn)(const float *, int64_t, const float *, int64_t, const float *, int64_t, const float *,
                         const int32_t *, const int32_t *, int, int, const dl_block_tables *, const dl_rope *,
                         const dl_paged_kv *, float *, int64_t, float *, int64_t, float *, int64_t, int32_t *, dl_stream_t);
typedef int (*attn_fn)(const float *, int64_t, const dl_paged_kv *, const dl_block_tables *, const int32_t *,
                       const int32_t *, int, int, int, const int32_t *, int, float *, int64_t, float *, void *, size_t,
                       int32_t *, dl_stream_t);
typedef int (*select_fn)(const float *, int64_t, const dl_paged_kv *, const dl_block_tables *, const int32_t *, int, int,
                         int, int, int, int32_t *, int32_t *, dl_stream_t);

static append_fn f_append;
static attn_fn f_attn;
static select_fn f_select;
static PyObject *t_f32, *t_i32, *t_u8;                        /* torch.float32, torch.int32, torch.uint8 */
static PyObject *n_dtype, *n_device, *n_get_device, *n_shape, *n_stride, *n_data_ptr;

/* ---- one tensor */

typedef struct {
    void *p;
    int dim;
    int64_t size[4], stride[4];
} tensor;

/* The whole number an attribute's call returns. */
static int call_number(PyObject *t, PyObject *name, long long *out)
{
    PyObject *r = PyObject_CallMethodNoArgs(t, name);
    if (!r) return -1;
    *out = PyLong_AsLongLong(r);
    Py_DECREF(r);
    return *out == -1 && PyErr_Occurred() ? -1 : 0;
}

static int numbers_of(PyObject *tuple, int64_t *out, int *n, const char *name)
{
    if (!tuple) return -1;
    if (!PyTuple_Check(tuple) || PyTuple_GET_SIZE(tuple) > 4) {
        PyErr_Format(PyExc_ValueError, "%s has more dimensions than any argument may have", name);
        return -1;
    }
    *n = (int)PyTuple_GET_SIZE(tuple);
    for (int i = 0; i < *n; ++i) {
        out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
        if (out[i] == -1 && PyErr_Occurred()) return -1;
    }
    return 0;
}

/* t on CUDA device `dev` with that dtype; 1, 0 for None where that may be (p = NULL), -1 with an error set. */
static int get(PyObject *t, long dev, PyObject *dtype, const char *name, int may_be_none, tensor *out)
{
    out->p = NULL;
    out->dim = 0;
    if (t == Py_None && may_be_none) return 0;
    PyObject *d = PyObject_GetAttr(t, n_dtype);
    if (!d) return -1;
    Py_DECREF(d);
    if (d != dtype) {
        PyErr_Format(PyExc_TypeError, "%s must be %S, got %S", name, dtype, d);
        return -1;
    }
    long long where, addr;
    if (call_number(t, n_get_device, &where)) return -1;
    if (where != dev || dev < 0) {
        PyObject *w = PyObject_GetAttr(t, n_device);
        if (w) PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor on the cache's device, got one on %S", name, w);
        Py_XDECREF(w);
        return -1;
    }
    if (call_number(t, n_data_ptr, &addr)) return -1;
    out->p = (void *)(intptr_t)addr;
    PyObject *s = PyObject_GetAttr(t, n_shape);
    int rc = numbers_of(s, out->size, &out->dim, name);
    Py_XDECREF(s);
    if (rc) return -1;
    s = PyObject_CallMethodNoArgs(t, n_stride);
    int n;
    rc = numbers_of(s, out->stride, &n, name);
    Py_XDECREF(s);
    return rc ? -1 : 1;
}

static int dense(const tensor *t)
{
    int64_t want = 1;
    for (int i = t->dim - 1; i >= 0; --i) {
        if (t->size[i] > 1 && t->stride[i] != want) return 0;
        want *= t->size[i] > 1 ? t->size[i] : 1;
    }
    return 1;
}

/* ---- arguments */

/* f32 [rows][>= width] rows with unit inner stride. */
static int get_rows(PyObject *o, long dev, int64_t rows, int64_t width, const char *name, int may_be_none, float **p,
                    int64_t *stride)
{
    tensor t;
    const int r = get(o, dev, t_f32, name, may_be_none, &t);
    *p = (float *)t.p;
    *stride = 0;
    if (r <= 0) return r;
    if (t.dim != 2 || t.size[0] != rows || t.size[1] < width || (t.size[1] > 1 && t.stride[1] != 1)) {
        PyErr_Format(PyExc_ValueError, "%s must be [%lld][>= %lld] rows with unit inner stride", name, (long long)rows,
                     (long long)width);
        return -1;
    }
    /* a single row's stride means nothing and torch may give it any value */
    *stride = rows > 1 ? t.stride[0] : (width + 3) / 4 * 4;
    return 1;
}

static int get_ints(PyObject *o, long dev, int64_t n, const char *name, int may_be_none, const int32_t **p)
{
    tensor t;
    const int r = get(o, dev, t_i32, name, may_be_none, &t);
    *p = (const int32_t *)t.p;
    if (r <= 0) return r;
    if (t.dim != 1 || t.size[0] < n || !dense(&t)) {
        PyErr_Format(PyExc_ValueError, "%s must be a dense vector of at least %lld int32", name, (long long)n);
        return -1;
    }
    return 1;
}

static int get_tables(PyObject *o, long dev, dl_block_tables *out)
{
    tensor t;
    if (get(o, dev, t_i32, "tables", 0, &t) < 0) return -1;
    if (t.dim != 2 || (t.size[1] > 1 && t.stride[1] != 1) || t.size[0] > INT32_MAX || t.size[1] > INT32_MAX) {
        PyErr_SetString(PyExc_ValueError, "tables must be [sequences][width] int32 with unit inner stride");
        return -1;
    }
    out->pages = (const int32_t *)t.p;
    out->stride = t.size[0] > 1 ? t.stride[0] : (t.size[1] > 1 ? t.size[1] : 1);
    out->n_seqs = (int)t.size[0];
    out->width = (int)t.size[1];
    return 0;
}

static int get_status(PyObject *o, long dev, int32_t **p)
{
    tensor t;
    const int r = get(o, dev, t_i32, "status", 1, &t);
    *p = (int32_t *)t.p;
    if (r <= 0) return r;
    for (int i = 0; i < t.dim; ++i)
        if (t.size[i] < 1) {
            PyErr_SetString(PyExc_ValueError, "status must hold one int32");
            return -1;
        }
    return 1;
}

/* A dense tensor of exactly this shape (n numbers). */
static int get_exact(PyObject *o, long dev, PyObject *dtype, const char *name, int may_be_none, int n, const int64_t *shape,
                     void **p)
{
    tensor t;
    const int r = get(o, dev, dtype, name, may_be_none, &t);
    *p = t.p;
    if (r <= 0) return r;
    int ok = t.dim == n && dense(&t);
    for (int i = 0; ok && i < n; ++i) ok = t.size[i] == shape[i];
    if (ok) return 1;
    PyErr_Format(PyExc_ValueError, n == 1   ? "%s must be a dense vector of %lld"
                                   : n == 2 ? "%s must be contiguous [%lld][%lld]"
                                            : "%s must be contiguous [%lld][%lld][%lld]",
                 name, (long long)shape[0], n > 1 ? (long long)shape[1] : 0, n > 2 ? (long long)shape[2] : 0);
    return -1;
}

static int get_int(PyObject *o, const char *name, int *out)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) return -1;
    if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_Format(PyExc_ValueError, "%s = %lld is past 32 bits", name, v);
        return -1;
    }
    *out = (int)v;
    return 0;
}

/* Rows of a 2-D tensor (its other checks follow when it is read). */
static int count_rows(PyObject *o, int64_t *rows)
{
    PyObject *s = PyObject_GetAttr(o, n_shape);
    int64_t size[4];
    int n;
    const int rc = numbers_of(s, size, &n, "q");
    Py_XDECREF(s);
    if (rc) return -1;
    if (n != 2 || size[0] > INT32_MAX) {
        PyErr_SetString(PyExc_ValueError, "q must be 2-D rows");
        return -1;
    }
    *rows = size[0];
    return 0;
}

/* The handle every call starts with: (cache address, device, n_kv, head_dim). */
typedef struct {
    const dl_paged_kv *kv;
    long dev;
} handle;
static int get_handle(PyObject *addr, PyObject *dev, handle *h)
{
    h->kv = (const dl_paged_kv *)PyLong_AsVoidPtr(addr);
    if (!h->kv && PyErr_Occurred()) return -1;
    h->dev = PyLong_AsLong(dev);
    return h->dev == -1 && PyErr_Occurred() ? -1 : 0;
}

static int arity(const char *f, Py_ssize_t n, Py_ssize_t want)
{
    if (n == want) return 0;
    PyErr_Format(PyExc_TypeError, "%s: %zd arguments, %zd wanted", f, n, want);
    return -1;
}

/* ---- the calls: their status, or an exception */

/* append(kv, dev, q, k, v, pos, tables, rope, rope_table, n_q, row_seq, bias, q_out, k_out, v_out, status, stream) */
static PyObject *py_append(PyObject *self, PyObject *const *a, Py_ssize_t nargs)
{
    (void)self;
    handle h;
    int n_q;
    int64_t rows, qs, ks, vs, qos, kos, vos;
    float *q, *k, *v, *qo, *ko, *vo;
    void *bias;
    const int32_t *pos, *seq;
    int32_t *status;
    dl_block_tables t;
    tensor rt;
    if (arity("append", nargs, 17) || get_handle(a[0], a[1], &h) || get_int(a[9], "n_q", &n_q) || count_rows(a[2], &rows))
        return NULL;
    const dl_rope *rope = (const dl_rope *)PyLong_AsVoidPtr(a[7]);
    if (!rope) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no rope");
        return NULL;
    }
    const int64_t qw = (int64_t)n_q * h.kv->head_dim, kw = (int64_t)h.kv->n_kv * h.kv->head_dim, bw = qw + 2 * kw;
    if (get_rows(a[2], h.dev, rows, qw, "q", 0, &q, &qs) < 0 || get_rows(a[3], h.dev, rows, kw, "k", 0, &k, &ks) < 0 ||
        get_rows(a[4], h.dev, rows, kw, "v", 0, &v, &vs) < 0 || get_ints(a[5], h.dev, rows, "pos", 0, &pos) < 0 ||
        get_tables(a[6], h.dev, &t) || (rope->rot_dim && get(a[8], h.dev, t_f32, "rope.table", 0, &rt) < 0) ||
        get_ints(a[10], h.dev, rows, "row_seq", 1, &seq) < 0 ||
        get_exact(a[11], h.dev, t_f32, "bias", 1, 1, &bw, &bias) < 0 ||
        get_rows(a[12], h.dev, rows, qw, "q_out", 1, &qo, &qos) < 0 ||
        get_rows(a[13], h.dev, rows, kw, "k_out", 1, &ko, &kos) < 0 ||
        get_rows(a[14], h.dev, rows, kw, "v_out", 1, &vo, &vos) < 0 || get_status(a[15], h.dev, &status) < 0)
        return NULL;
    dl_stream_t stream = PyLong_AsVoidPtr(a[16]);
    if (!stream && PyErr_Occurred()) return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f_append(q, qs, k, ks, v, vs, (const float *)bias, pos, seq, (int)rows, n_q, &t, rope, h.kv, qo, qos, ko, kos, vo,
                  vos, status, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* attn(kv, dev, q, tables, seqlen, workspace, n_q, out, lse, row_begin, max_rows, pages, status, stream) */
static PyObject *py_attn(PyObject *self, PyObject *const *a, Py_ssize_t nargs)
{
    (void)self;
    handle h;
    int n_q, max_rows, n_list = 0;
    int64_t rows, qs, os;
    float *q, *out;
    void *lse;
    const int32_t *seqlen, *begin, *pages;
    int32_t *status;
    dl_block_tables t;
    tensor ws, pg;
    if (arity("attn", nargs, 14) || get_handle(a[0], a[1], &h) || get_int(a[6], "n_q", &n_q) ||
        get_int(a[10], "max_rows", &max_rows) || count_rows(a[2], &rows))
        return NULL;
    const int64_t width = (int64_t)n_q * h.kv->head_dim, lse_shape[2] = {rows, n_q};
    if (get_rows(a[2], h.dev, rows, width, "q", 0, &q, &qs) < 0 || get_tables(a[3], h.dev, &t) ||
        get_ints(a[4], h.dev, t.n_seqs, "seqlen", 0, &seqlen) < 0 || get(a[5], h.dev, t_u8, "workspace", 0, &ws) < 0 ||
        get_rows(a[7], h.dev, rows, width, "out", 0, &out, &os) < 0 ||
        get_exact(a[8], h.dev, t_f32, "lse", 1, 2, lse_shape, &lse) < 0 ||
        get_ints(a[9], h.dev, (int64_t)t.n_seqs + 1, "row_begin", 1, &begin) < 0)
        return NULL;
    if (ws.dim != 1 || !dense(&ws)) {
        PyErr_SetString(PyExc_ValueError, "workspace must be a dense vector of bytes");
        return NULL;
    }
    const int listed = get(a[11], h.dev, t_i32, "pages", 1, &pg);
    if (listed < 0) return NULL;
    pages = (const int32_t *)pg.p;
    if (listed) {
        if (pg.dim != 3 || pg.size[0] != rows || pg.size[1] != h.kv->n_kv || pg.size[2] < 1 ||
            pg.size[2] > INT32_MAX || !dense(&pg)) {
            PyErr_Format(PyExc_ValueError, "pages must be contiguous [%lld][%d][>= 1]", (long long)rows, h.kv->n_kv);
            return NULL;
        }
        n_list = (int)pg.size[2];
    }
    if (get_status(a[12], h.dev, &status) < 0) return NULL;
    dl_stream_t stream = PyLong_AsVoidPtr(a[13]);
    if (!stream && PyErr_Occurred()) return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f_attn(q, qs, h.kv, &t, seqlen, begin, (int)rows, max_rows, n_q, pages, n_list, out, os, (float *)lse, ws.p,
                (size_t)ws.size[0], status, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* select(kv, dev, q, tables, seqlen, n_q, pages, top_k, n_sink, n_local, status, stream) */
static PyObject *py_select(PyObject *self, PyObject *const *a, Py_ssize_t nargs)
{
    (void)self;
    handle h;
    int n_q, top_k, sink, local;
    int64_t rows, qs;
    float *q;
    void *pages;
    const int32_t *seqlen;
    int32_t *status;
    dl_block_tables t;
    if (arity("select", nargs, 12) || get_handle(a[0], a[1], &h) || get_int(a[5], "n_q", &n_q) ||
        get_int(a[7], "top_k", &top_k) || get_int(a[8], "n_sink", &sink) || get_int(a[9], "n_local", &local) ||
        count_rows(a[2], &rows))
        return NULL;
    const int64_t shape[3] = {rows, h.kv->n_kv, (int64_t)top_k + sink + local};
    if (get_rows(a[2], h.dev, rows, (int64_t)n_q * h.kv->head_dim, "q", 0, &q, &qs) < 0 || get_tables(a[3], h.dev, &t) ||
        get_ints(a[4], h.dev, t.n_seqs, "seqlen", 0, &seqlen) < 0 ||
        get_exact(a[6], h.dev, t_i32, "pages", 0, 3, shape, &pages) < 0 || get_status(a[10], h.dev, &status) < 0)
        return NULL;
    dl_stream_t stream = PyLong_AsVoidPtr(a[11]);
    if (!stream && PyErr_Occurred()) return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f_select(q, qs, h.kv, &t, seqlen, (int)rows, n_q, top_k, sink, local, (int32_t *)pages, status, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* bind(append, attn, select, float32, int32, uint8): the library's functions by address and torch's dtypes */
static PyObject *py_bind(PyObject *self, PyObject *args)
{
    (void)self;
    PyObject *x, *y, *z, *f, *i, *u;
    if (!PyArg_ParseTuple(args, "OOOOOO", &x, &y, &z, &f, &i, &u)) return NULL;
    f_append = (append_fn)PyLong_AsVoidPtr(x);
    f_attn = (attn_fn)PyLong_AsVoidPtr(y);
    f_select = (select_fn)PyLong_AsVoidPtr(z);
    if (!f_append || !f_attn || !f_select) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null function");
        return NULL;
    }
    Py_INCREF(f);
    Py_INCREF(i);
    Py_INCREF(u);
    Py_XDECREF(t_f32);
    Py_XDECREF(t_i32);
    Py_XDECREF(t_u8);
    t_f32 = f;
    t_i32 = i;
    t_u8 = u;
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"append", (PyCFunction)(void (*)(void))py_append, METH_FASTCALL, NULL},
    {"attn", (PyCFunction)(void (*)(void))py_attn, METH_FASTCALL, NULL},
    {"select", (PyCFunction)(void (*)(void))py_select, METH_FASTCALL, NULL},
    {"bind", py_bind, METH_VARARGS, NULL},
    {NULL, NULL, 0, NULL},
};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_call", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__paged_call(void)
{
    n_dtype = PyUnicode_InternFromString("dtype");
    n_device = PyUnicode_InternFromString("device");
    n_get_device = PyUnicode_InternFromString("get_device");
    n_shape = PyUnicode_InternFromString("shape");
    n_stride = PyUnicode_InternFromString("stride");
    n_data_ptr = PyUnicode_InternFromString("data_ptr");
    if (!n_dtype || !n_device || !n_get_device || !n_shape || !n_stride || !n_data_ptr) return NULL;
    return PyModule_Create(&module);
}
