/*
 * marshal.c -- the argument checks of the dense network's Python binding, as a
 * CPython extension (dense.py).  A layer on a few rows takes the GPU 2 us; with
 * its checks and the ctypes call in Python the host needed 8 us for it.
 *
 * Each function takes the tensors and numbers of one entry point of
 * include/dlrm_dense.h, checks shapes, dtypes and strides, then that every tensor
 * is on the current device (TypeError, ValueError), calls the entry point through
 * the address bind() was given and returns its status.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <limits.h>

#include "dlrm_dense.h"

static PyObject *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_nbytes, *s_get_device, *s_is_contiguous;
/* torch's dtypes: fp32, fp16, bf16 (their codes are the indices), int32, int64 */
enum { F32, F16, BF16, I32, I64, N_TYPES };
static PyObject* types[N_TYPES];
static PyObject *get_device, *get_raw_stream;

static struct {
    dlrm_status (*dropout_fwd)(const void*, int64_t, const void*, int64_t, dlrm_dtype, int, int, double, const uint64_t*,
                               void*, int64_t, void*);
    dlrm_status (*dropout_bwd)(const void*, int64_t, dlrm_dtype, int, int, double, const uint64_t*, void*, int64_t, void*);
    dlrm_status (*linear_fwd)(const void*, int64_t, const void*, int64_t, const float*, const void*, int64_t, dlrm_dtype,
                              int, int, int, dlrm_act, double, const uint64_t*, void*, int64_t, void*, int64_t, void*,
                              size_t, uint32_t*, void*);
    dlrm_status (*linear_bwd)(const void*, int64_t, const void*, int64_t, const void*, int64_t, const void*, int64_t,
                              dlrm_dtype, int, int, int, dlrm_act, double, const uint64_t*, void*, int64_t, void*, int64_t,
                              float*, void*, size_t, uint32_t*, void*);
    dlrm_status (*moe_fwd)(const void*, int64_t, const void*, const void*, const void*, const void*, int64_t, dlrm_dtype,
                           int, int, int, int, int, dlrm_act, int, void*, int64_t, int32_t*, float*, void*, size_t,
                           uint32_t*, void*);
} fn;

/* ------------------------------------------------------------------ tensors */
/* The tensor's sizes, which have to be nd; 0 with an exception set otherwise. */
static int sizes(PyObject* t, const char* name, int nd, int64_t* out)
{
    PyObject* s = PyObject_GetAttr(t, s_shape);
    if (!s) return 0;
    int ok = PyTuple_Check(s) && PyTuple_GET_SIZE(s) == nd;
    for (int i = 0; ok && i < nd; ++i) {
        out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(s, i));
        if (out[i] > INT32_MAX) {
            PyErr_Format(PyExc_ValueError, "%s has a size past 2^31", name);
            Py_DECREF(s);
            return 0;
        }
    }
    if (!ok && !PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "%s has shape %S, not %d sizes", name, s, nd);
    Py_DECREF(s);
    return ok && !PyErr_Occurred();
}

static int has_type(PyObject* t, const char* name, PyObject* type)
{
    PyObject* d = PyObject_GetAttr(t, s_dtype);
    if (!d) return 0;
    const int ok = d == type;
    if (!ok) PyErr_Format(PyExc_TypeError, "%s is %S, not %S", name, d, type);
    Py_DECREF(d);
    return ok;
}

/* The code of the tensor's element type; -1 with an exception set. */
static int type_code(PyObject* t)
{
    PyObject* d = PyObject_GetAttr(t, s_dtype);
    if (!d) return -1;
    int code = 0;
    while (code <= BF16 && d != types[code]) ++code;
    if (code > BF16) PyErr_Format(PyExc_TypeError, "unsupported dtype %S", d);
    Py_DECREF(d);
    return code > BF16 ? -1 : code;
}

static int address(PyObject* t, void** p)
{
    PyObject* a = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!a) return 0;
    *p = PyLong_AsVoidPtr(a);
    Py_DECREF(a);
    return !PyErr_Occurred();
}

/* Checks an nd-dimensional argument: sizes, dtype, and strides: contiguous, or with ld
   (nd == 2) unit column stride, the row distance to *ld.  None: NULL. */
static int argument(PyObject* t, const char* name, PyObject* type, int nd, const int64_t* want, void** p, int64_t* ld)
{
    *p = NULL;
    if (ld) *ld = 0;
    if (t == Py_None) return 1;
    if (!has_type(t, name, type)) return 0;
    int64_t got[3];
    if (!sizes(t, name, nd, got)) return 0;
    for (int i = 0; i < nd; ++i)
        if (got[i] != want[i]) {
            PyErr_Format(PyExc_ValueError, "size %d of %s is %lld, not %lld", i, name, (long long)got[i], (long long)want[i]);
            return 0;
        }
    PyObject* s = PyObject_CallMethodNoArgs(t, s_stride);
    if (!s) return 0;
    int64_t next = 1;
    int ok = PyTuple_Check(s) && PyTuple_GET_SIZE(s) == nd, empty = 0;
    for (int i = 0; i < nd; ++i) empty |= got[i] == 0;
    for (int i = nd - 1; ok && i >= 0; --i) {
        const int64_t v = PyLong_AsLongLong(PyTuple_GET_ITEM(s, i));
        if (ld && i == 0) *ld = v;
        else ok = empty || got[i] == 1 || v == next;
        next *= got[i];
    }
    Py_DECREF(s);
    if (!ok) {
        PyErr_Format(PyExc_ValueError, ld ? "%s must have unit column stride" : "%s must be contiguous", name);
        return 0;
    }
    return address(t, p);
}

static int matrix(PyObject* t, const char* name, PyObject* type, int64_t rows, int64_t cols, void** p, int64_t* ld)
{
    const int64_t want[2] = {rows, cols};
    return argument(t, name, type, 2, want, p, ld);
}

static int vector(PyObject* t, const char* name, PyObject* type, int64_t n, void** p)
{
    return argument(t, name, type, 1, &n, p, NULL);
}

static int workspace(PyObject* t, void** p, size_t* bytes)
{
    *p = NULL;
    *bytes = 0;
    if (t == Py_None) return 1;
    PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (!c) return 0;
    const int contiguous = PyObject_IsTrue(c);
    Py_DECREF(c);
    if (contiguous < 0) return 0;
    if (!contiguous) {   /* an expanded tensor has fewer bytes than it says */
        PyErr_SetString(PyExc_ValueError, "workspace must be contiguous");
        return 0;
    }
    PyObject* n = PyObject_GetAttr(t, s_nbytes);
    if (!n) return 0;
    *bytes = PyLong_AsSize_t(n);
    Py_DECREF(n);
    return !PyErr_Occurred() && address(t, p);
}

static int status_word(PyObject* t, void** p)
{
    *p = NULL;
    if (t == Py_None) return 1;
    if (PyLong_Check(t)) {
        *p = PyLong_AsVoidPtr(t);
        return !PyErr_Occurred();
    }
    PyObject* n = PyObject_GetAttr(t, s_nbytes);
    if (!n) return 0;
    const size_t bytes = PyLong_AsSize_t(n);
    Py_DECREF(n);
    if (PyErr_Occurred()) return 0;
    if (bytes < 4) {
        PyErr_SetString(PyExc_ValueError, "status has fewer than 4 bytes");
        return 0;
    }
    return address(t, p);
}

/* The last of a call's checks: its tensors (the first n of t that are not None, nor
   numbers: addresses) are on the current device.  Then the stream's handle; None: torch's
   current stream on that device. */
static int where(PyObject* const* t, const char* const* names, int n, PyObject* on, void** p)
{
    PyObject* d = NULL;
    long current = 0;
    for (int i = 0; i < n; ++i) {
        if (t[i] == Py_None || !names[i] || PyLong_Check(t[i])) continue;
        PyObject* o = PyObject_CallMethodNoArgs(t[i], s_get_device);
        if (!o) goto bad;
        const long at = PyLong_AsLong(o);
        Py_DECREF(o);
        if (at == -1 && PyErr_Occurred()) goto bad;
        if (at < 0) {
            PyErr_Format(PyExc_ValueError, "%s is not on a CUDA device", names[i]);
            goto bad;
        }
        if (!d) {
            d = PyObject_CallNoArgs(get_device);
            if (!d) return 0;
            current = PyLong_AsLong(d);
            if (current == -1 && PyErr_Occurred()) goto bad;
        }
        if (at != current) {
            PyErr_Format(PyExc_ValueError, "%s is on device %ld, not on the current one (%ld)", names[i], at, current);
            goto bad;
        }
    }
    if (on != Py_None) {
        Py_XDECREF(d);
        *p = PyLong_AsVoidPtr(on);
        return !PyErr_Occurred();
    }
    if (!d && !(d = PyObject_CallNoArgs(get_device))) return 0;
    PyObject* s = PyObject_CallOneArg(get_raw_stream, d);
    Py_DECREF(d);
    if (!s) return 0;
    *p = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    return !PyErr_Occurred();
bad:
    Py_XDECREF(d);
    return 0;
}

static int number(PyObject* t, int* v)
{
    const long long l = PyLong_AsLongLong(t);
    if (l == -1 && PyErr_Occurred()) return 0;
    if (l < INT_MIN || l > INT_MAX) {
        PyErr_Format(PyExc_ValueError, "act is %lld", l);
        return 0;
    }
    *v = (int)l;
    return 1;
}

static int real(PyObject* t, double* v)
{
    *v = PyFloat_AsDouble(t);
    return !PyErr_Occurred();
}

static int count(Py_ssize_t got, Py_ssize_t want)
{
    if (got == want) return 1;
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", got, want);
    return 0;
}

/* -------------------------------------------------------------- entry points */
/* x, residual, y, p, rng, stream */
static PyObject* dropout_fwd(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    int64_t mn[2], ldx, ldr, ldy;
    void *x, *r, *y, *rng, *st;
    double p;
    int c;
    static const char* const names[] = {"x", "residual", "y", NULL, "rng"};
    if (!count(n, 6) || (c = type_code(a[0])) < 0 || !sizes(a[0], "x", 2, mn) ||
        !matrix(a[0], "x", types[c], mn[0], mn[1], &x, &ldx) || !matrix(a[1], "residual", types[c], mn[0], mn[1], &r, &ldr) ||
        !matrix(a[2], "y", types[c], mn[0], mn[1], &y, &ldy) || !real(a[3], &p) ||
        !vector(a[4], "rng", types[I64], 2, &rng) || !where(a, names, 5, a[5], &st))
        return NULL;
    return PyLong_FromLong(fn.dropout_fwd(x, ldx, r, ldr, (dlrm_dtype)c, (int)mn[0], (int)mn[1], p, rng, y, ldy, st));
}

/* grad_y, grad_x, p, rng, stream */
static PyObject* dropout_bwd(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    int64_t mn[2], ldg, ldx;
    void *g, *x, *rng, *st;
    double p;
    int c;
    static const char* const names[] = {"grad_y", "grad_x", NULL, "rng"};
    if (!count(n, 5) || (c = type_code(a[0])) < 0 || !sizes(a[0], "grad_y", 2, mn) ||
        !matrix(a[0], "grad_y", types[c], mn[0], mn[1], &g, &ldg) || !matrix(a[1], "grad_x", types[c], mn[0], mn[1], &x, &ldx) ||
        !real(a[2], &p) || !vector(a[3], "rng", types[I64], 2, &rng) || !where(a, names, 4, a[4], &st))
        return NULL;
    return PyLong_FromLong(fn.dropout_bwd(g, ldg, (dlrm_dtype)c, (int)mn[0], (int)mn[1], p, rng, x, ldx, st));
}

/* x, w, bias, residual, y, pre, act, p, rng, workspace, status, stream */
static PyObject* linear_fwd(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    int64_t mk[2], nk[2], ldx, ldw, ldr, ldy, ldp;
    void *x, *w, *b, *r, *y, *z, *rng, *ws, *status, *st;
    size_t bytes;
    double p;
    int c, act;
    static const char* const names[] = {"x", "w", "bias", "residual", "y", "pre", NULL, NULL, "rng", "workspace", "status"};
    if (!count(n, 12) || (c = type_code(a[0])) < 0 || !sizes(a[0], "x", 2, mk) || !sizes(a[1], "w", 2, nk)) return NULL;
    PyObject* t = types[c];
    const int64_t M = mk[0], K = mk[1], N = nk[0];
    if (!matrix(a[0], "x", t, M, K, &x, &ldx) || !matrix(a[1], "w", t, N, K, &w, &ldw) ||
        !vector(a[2], "bias", types[F32], N, &b) || !matrix(a[3], "residual", t, M, N, &r, &ldr) ||
        !matrix(a[4], "y", t, M, N, &y, &ldy) || !matrix(a[5], "pre", t, M, N, &z, &ldp) || !number(a[6], &act) ||
        !real(a[7], &p) || !vector(a[8], "rng", types[I64], 2, &rng) || !workspace(a[9], &ws, &bytes) ||
        !status_word(a[10], &status) || !where(a, names, 11, a[11], &st))
        return NULL;
    return PyLong_FromLong(fn.linear_fwd(x, ldx, w, ldw, b, r, ldr, (dlrm_dtype)c, (int)M, (int)N, (int)K, (dlrm_act)act, p,
                                         rng, y, ldy, z, ldp, ws, bytes, status, st));
}

/* grad_y, x, w, pre, grad_x, grad_w, grad_bias, act, p, rng, workspace, status, stream */
static PyObject* linear_bwd(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    int64_t mk[2], nk[2], ldg, ldx, ldw, ldp, lddx, lddw;
    void *g, *x, *w, *z, *dx, *dw, *db, *rng, *ws, *status, *st;
    size_t bytes;
    double p;
    int c, act;
    static const char* const names[] = {"grad_y", "x",  "w",  "pre", "grad_x",    "grad_w",
                                        "grad_bias", NULL, NULL, "rng", "workspace", "status"};
    if (!count(n, 13) || (c = type_code(a[1])) < 0 || !sizes(a[1], "x", 2, mk) || !sizes(a[2], "w", 2, nk)) return NULL;
    PyObject* t = types[c];
    const int64_t M = mk[0], K = mk[1], N = nk[0];
    if (!matrix(a[0], "grad_y", t, M, N, &g, &ldg) || !matrix(a[1], "x", t, M, K, &x, &ldx) ||
        !matrix(a[2], "w", t, N, K, &w, &ldw) || !matrix(a[3], "pre", t, M, N, &z, &ldp) ||
        !matrix(a[4], "grad_x", t, M, K, &dx, &lddx) || !matrix(a[5], "grad_w", t, N, K, &dw, &lddw) ||
        !vector(a[6], "grad_bias", types[F32], N, &db) || !number(a[7], &act) || !real(a[8], &p) ||
        !vector(a[9], "rng", types[I64], 2, &rng) || !workspace(a[10], &ws, &bytes) || !status_word(a[11], &status) ||
        !where(a, names, 12, a[12], &st))
        return NULL;
    return PyLong_FromLong(fn.linear_bwd(g, ldg, x, ldx, w, ldw, z, ldp, (dlrm_dtype)c, (int)M, (int)N, (int)K,
                                         (dlrm_act)act, p, rng, dx, lddx, dw, lddw, db, ws, bytes, status, st));
}

/* x, w_router, w1, w2, residual, y, ids, probs, act, gated, workspace, status, stream */
static PyObject* moe_fwd(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    int64_t th[2], eh[2], ehi[3], tk[2], ldx, ldr, ldy;
    void *x, *wr, *w1, *w2, *r, *y, *ids, *probs, *ws, *status, *st;
    size_t bytes;
    int c, act, gated;
    static const char* const names[] = {"x",   "w_router", "w1", "w2", "residual",  "y",
                                        "ids", "probs",    NULL, NULL, "workspace", "status"};
    if (!count(n, 13) || (c = type_code(a[0])) < 0 || !sizes(a[0], "x", 2, th) || !sizes(a[1], "w_router", 2, eh) ||
        !sizes(a[3], "w2", 3, ehi) || !sizes(a[6], "ids", 2, tk) || (gated = PyObject_IsTrue(a[9])) < 0)
        return NULL;
    PyObject* t = types[c];
    const int64_t T = th[0], H = th[1], E = eh[0], I = ehi[2], k = tk[1];
    const int64_t router[2] = {E, H}, first[3] = {E, gated ? 2 * I : I, H}, second[3] = {E, H, I}, choice[2] = {T, k};
    if (!matrix(a[0], "x", t, T, H, &x, &ldx) || !argument(a[1], "w_router", t, 2, router, &wr, NULL) ||
        !argument(a[2], "w1", t, 3, first, &w1, NULL) || !argument(a[3], "w2", t, 3, second, &w2, NULL) ||
        !matrix(a[4], "residual", t, T, H, &r, &ldr) || !matrix(a[5], "y", t, T, H, &y, &ldy) ||
        !argument(a[6], "ids", types[I32], 2, choice, &ids, NULL) ||
        !argument(a[7], "probs", types[F32], 2, choice, &probs, NULL) || !number(a[8], &act) ||
        !workspace(a[10], &ws, &bytes) || !status_word(a[11], &status) || !where(a, names, 12, a[12], &st))
        return NULL;
    return PyLong_FromLong(fn.moe_fwd(x, ldx, wr, w1, w2, r, ldr, (dlrm_dtype)c, (int)T, (int)H, (int)I, (int)E, (int)k,
                                      (dlrm_act)act, gated, y, ldy, ids, probs, ws, bytes, status, st));
}

/* bind((fp32, fp16, bf16, int32, int64 dtypes), current_device, current_raw_stream, (addresses of
   dropout_fwd, dropout_bwd, linear_fwd, linear_bwd, moe_fwd)) */
static PyObject* bind(PyObject* self, PyObject* args)
{
    PyObject *dtypes, *device, *raw, *at;
    if (!PyArg_ParseTuple(args, "O!OOO!", &PyTuple_Type, &dtypes, &device, &raw, &PyTuple_Type, &at)) return NULL;
    if (!count(PyTuple_GET_SIZE(dtypes), N_TYPES) || !count(PyTuple_GET_SIZE(at), 5)) return NULL;
    void* p[5];
    for (int i = 0; i < 5; ++i) {
        p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(at, i));
        if (PyErr_Occurred()) return NULL;
    }
    for (int i = 0; i < N_TYPES; ++i) Py_XSETREF(types[i], Py_NewRef(PyTuple_GET_ITEM(dtypes, i)));
    Py_XSETREF(get_device, Py_NewRef(device));
    Py_XSETREF(get_raw_stream, Py_NewRef(raw));
    *(void**)&fn.dropout_fwd = p[0];
    *(void**)&fn.dropout_bwd = p[1];
    *(void**)&fn.linear_fwd = p[2];
    *(void**)&fn.linear_bwd = p[3];
    *(void**)&fn.moe_fwd = p[4];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, NULL},
    {"dropout_fwd", (PyCFunction)(void (*)(void))dropout_fwd, METH_FASTCALL, NULL},
    {"dropout_bwd", (PyCFunction)(void (*)(void))dropout_bwd, METH_FASTCALL, NULL},
    {"linear_fwd", (PyCFunction)(void (*)(void))linear_fwd, METH_FASTCALL, NULL},
    {"linear_bwd", (PyCFunction)(void (*)(void))linear_bwd, METH_FASTCALL, NULL},
    {"moe_fwd", (PyCFunction)(void (*)(void))moe_fwd, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void)
{
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_nbytes = PyUnicode_InternFromString("nbytes");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    if (!s_dtype || !s_shape || !s_stride || !s_data_ptr || !s_nbytes || !s_get_device || !s_is_contiguous) return NULL;
    return PyModule_Create(&module);
}
