/*
 * marshal.c -- the argument checks of the dense network's Python binding, as a
 * CPython extension (dense.py).  A layer on a few rows takes the GPU 2 us; with
 * its checks and the ctypes call in Python the host needed 8 us for it.
 *
 * Each function takes the tensors and numbers of one entry point of
 * include/dlrm_dense.h or dlrm_block.h, checks shapes, dtypes and strides, then that every tensor
 * is on the current device (TypeError, ValueError), calls the entry point through
 * the address bind() was given and returns its status.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <limits.h>

#include "dlrm_block.h"

static PyObject *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_nbytes, *s_get_device, *s_is_contiguous;
/* torch's dtypes: fp32, fp16, bf16 (their codes are the indices), int32, int64; uint8 comes with bind_block */
enum { F32, F16, BF16, I32, I64, N_TYPES, U8 = N_TYPES, N_ALL };
static PyObject* types[N_ALL];
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

/* ------------------------------------------------------- residual blocks (dlrm_block.h) */
static struct {
    dlrm_status (*block_norm_fwd)(const void*, int64_t, const void*, int64_t, int, const void*, int64_t, const float*,
                                  const float*, const float*, const float*, const float*, dlrm_dtype, int, int, dlrm_norm,
                                  dlrm_gate, double, void*, int64_t, void*, int64_t, float*, void*);
    dlrm_status (*block_norm_bwd)(const void*, int64_t, const void*, int64_t, const void*, int64_t, const void*, int64_t, int,
                                  const void*, int64_t, const float*, const float*, const float*, const float*, const float*,
                                  dlrm_dtype, int, int, dlrm_norm, dlrm_gate, void*, int64_t, void*, int64_t, void*, int64_t,
                                  float*, float*, float*, float*, float*, void*, size_t, void*);
    dlrm_status (*route_fwd)(const void*, int64_t, dlrm_dtype, int, int, int, int32_t*, float*, void*);
    dlrm_status (*route_bwd)(const float*, const int32_t*, const float*, dlrm_dtype, int, int, int, void*, int64_t, void*);
    dlrm_status (*expert_sort)(const int32_t*, int, int, int, int32_t*, int32_t*, int32_t*, void*, size_t, uint32_t*, void*);
    dlrm_status (*dispatch_fwd)(const void*, int64_t, const int32_t*, dlrm_dtype, int, int, int, int, void*, int64_t,
                                uint32_t*, void*);
    dlrm_status (*dispatch_bwd)(const void*, int64_t, const int32_t*, dlrm_dtype, int, int, int, int, void*, int64_t,
                                uint32_t*, void*);
    dlrm_status (*combine_fwd)(const void*, int64_t, const int32_t*, const float*, const void*, int64_t, dlrm_dtype, int, int,
                               int, int, void*, int64_t, uint32_t*, void*);
    dlrm_status (*combine_bwd)(const void*, int64_t, const void*, int64_t, const int32_t*, const float*, dlrm_dtype, int, int,
                               int, int, void*, int64_t, float*, uint32_t*, void*);
    dlrm_status (*pack8)(const void*, int64_t, dlrm_dtype, int, int, uint8_t*, int64_t, uint8_t*, void*);
    dlrm_status (*unpack8)(const uint8_t*, int64_t, const uint8_t*, dlrm_dtype, int, int, void*, int64_t, void*);
    dlrm_status (*linear_bwd8)(const void*, int64_t, const uint8_t*, int64_t, const uint8_t*, const void*, int64_t,
                               const uint8_t*, int64_t, const uint8_t*, dlrm_dtype, int, int, int, dlrm_act, double,
                               const uint64_t*, void*, int64_t, void*, int64_t, float*, void*, size_t, uint32_t*, void*);
} block;
#define N_BLOCK 12

/* The count of arguments, and that bind_block has been called: a library of before these entry points has none. */
static int ready(Py_ssize_t got, Py_ssize_t want)
{
    if (types[U8]) return count(got, want);
    PyErr_SetString(PyExc_RuntimeError, "the library was built before the residual blocks' entry points: build it again");
    return 0;
}

/* The first of n arguments that is a tensor; NULL with an exception set where none is. */
static PyObject* some(PyObject* const* t, int n, const char* names)
{
    for (int i = 0; i < n; ++i)
        if (t[i] != Py_None) return t[i];
    PyErr_Format(PyExc_ValueError, "none of %s is given", names);
    return NULL;
}

static int given(PyObject* t, const char* name)
{
    if (t != Py_None) return 1;
    PyErr_Format(PyExc_ValueError, "%s is None", name);
    return 0;
}

/* A code of an enumeration: what is out of a C int's range would be cut. */
static int code(PyObject* t, const char* name, int* v)
{
    const long long l = PyLong_AsLongLong(t);
    if (l == -1 && PyErr_Occurred()) return 0;
    if (l < INT_MIN || l > INT_MAX) {
        PyErr_Format(PyExc_ValueError, "%s is %lld", name, l);
        return 0;
    }
    *v = (int)l;
    return 1;
}

/* A gate [M][N] or [M][1]; *cols: its columns. */
static int gate_matrix(PyObject* t, const char* name, PyObject* type, const int64_t* mn, void** p, int64_t* ld, int64_t* cols)
{
    int64_t got[2];
    *cols = mn[1];
    if (t != Py_None) {
        if (!sizes(t, name, 2, got)) return 0;
        if (got[1] == 1) *cols = 1;
    }
    return matrix(t, name, type, mn[0], *cols, p, ld);
}

/* y, gate, residual, w_post, b_post, scale, w_pre, b_pre, r, h, stats, norm, gate_act, eps, stream */
static PyObject* block_norm_fwd(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    int64_t mn[2], ldy, ldg, ldres, ldr, ldh, cols;
    void *y, *g, *res, *v[5], *r, *h, *stats, *st;
    double eps;
    int c, norm, act;
    static const char* const names[] = {"y",     "gate",  "residual", "w_post", "b_post", "scale",
                                        "w_pre", "b_pre", "r",        "h",      "stats"};
    if (!ready(n, 15)) return NULL;
    PyObject *x = a[0] != Py_None ? a[0] : a[2], *t;
    if (!given(x, "residual") || (c = type_code(x)) < 0 || !sizes(x, x == a[0] ? "y" : "residual", 2, mn)) return NULL;
    t = types[c];
    if (!matrix(a[0], "y", t, mn[0], mn[1], &y, &ldy) || !gate_matrix(a[1], "gate", t, mn, &g, &ldg, &cols) ||
        !matrix(a[2], "residual", t, mn[0], mn[1], &res, &ldres))
        return NULL;
    for (int i = 0; i < 5; ++i)
        if (!vector(a[3 + i], names[3 + i], types[F32], mn[1], &v[i])) return NULL;
    const int64_t four[2] = {mn[0], 4};
    if (!matrix(a[8], "r", t, mn[0], mn[1], &r, &ldr) || !matrix(a[9], "h", t, mn[0], mn[1], &h, &ldh) ||
        !argument(a[10], "stats", types[F32], 2, four, &stats, NULL) || !code(a[11], "norm", &norm) ||
        !code(a[12], "gate_act", &act) || !real(a[13], &eps) || !where(a, names, 11, a[14], &st))
        return NULL;
    return PyLong_FromLong(block.block_norm_fwd(y, ldy, g, ldg, (int)cols, res, ldres, v[0], v[1], v[2], v[3], v[4],
                                                (dlrm_dtype)c, (int)mn[0], (int)mn[1], (dlrm_norm)norm, (dlrm_gate)act, eps,
                                                r, ldr, h, ldh, stats, st));
}

/* grad_r, grad_h, y, gate, r, stats, w_post, b_post, scale, w_pre, grad_y, grad_gate, grad_residual, grad_w_post,
   grad_b_post, grad_scale, grad_w_pre, grad_b_pre, norm, gate_act, workspace, stream */
static PyObject* block_norm_bwd(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    int64_t mn[2], ldgr, ldgh, ldy, ldg, ldr, ldgy, ldgg, ldgres, cols, gcols;
    void *gr, *gh, *y, *g, *r, *stats, *v[4], *gy, *gg, *gres, *o[5], *ws, *st;
    size_t bytes;
    int c, norm, act;
    static const char* const names[] = {"grad_r",      "grad_h",     "y",          "gate",      "r",
                                        "stats",       "w_post",     "b_post",     "scale",     "w_pre",
                                        "grad_y",      "grad_gate",  "grad_residual", "grad_w_post", "grad_b_post",
                                        "grad_scale",  "grad_w_pre", "grad_b_pre", NULL,        NULL,
                                        "workspace"};
    if (!ready(n, 22)) return NULL;
    PyObject* x = some(a, 2, "grad_r and grad_h");
    if (!x || (c = type_code(x)) < 0 || !sizes(x, x == a[0] ? "grad_r" : "grad_h", 2, mn)) return NULL;
    PyObject* t = types[c];
    const int64_t M = mn[0], N = mn[1], four[2] = {M, 4};
    if (!matrix(a[0], "grad_r", t, M, N, &gr, &ldgr) || !matrix(a[1], "grad_h", t, M, N, &gh, &ldgh) ||
        !matrix(a[2], "y", t, M, N, &y, &ldy) || !gate_matrix(a[3], "gate", t, mn, &g, &ldg, &cols) ||
        !matrix(a[4], "r", t, M, N, &r, &ldr) || !argument(a[5], "stats", types[F32], 2, four, &stats, NULL))
        return NULL;
    for (int i = 0; i < 4; ++i)
        if (!vector(a[6 + i], names[6 + i], types[F32], N, &v[i])) return NULL;
    gcols = cols;
    if (!matrix(a[10], "grad_y", t, M, N, &gy, &ldgy) || !matrix(a[11], "grad_gate", t, M, gcols, &gg, &ldgg) ||
        !matrix(a[12], "grad_residual", t, M, N, &gres, &ldgres))
        return NULL;
    for (int i = 0; i < 5; ++i)
        if (!vector(a[13 + i], names[13 + i], types[F32], N, &o[i])) return NULL;
    if (!code(a[18], "norm", &norm) || !code(a[19], "gate_act", &act) || !workspace(a[20], &ws, &bytes) ||
        !where(a, names, 21, a[21], &st))
        return NULL;
    return PyLong_FromLong(block.block_norm_bwd(gr, ldgr, gh, ldgh, y, ldy, g, ldg, (int)cols, r, ldr, stats, v[0], v[1],
                                                v[2], v[3], (dlrm_dtype)c, (int)M, (int)N, (dlrm_norm)norm, (dlrm_gate)act,
                                                gy, ldgy, gg, ldgg, gres, ldgres, o[0], o[1], o[2], o[3], o[4], ws, bytes,
                                                st));
}

/* logits, ids, probs, stream */
static PyObject* route_fwd(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    int64_t te[2], tk[2], ldl;
    void *l, *ids, *probs, *st;
    int c;
    static const char* const names[] = {"logits", "ids", "probs"};
    if (!ready(n, 4) || (c = type_code(a[0])) < 0 || !sizes(a[0], "logits", 2, te) || !sizes(a[1], "ids", 2, tk)) return NULL;
    const int64_t choice[2] = {te[0], tk[1]};
    if (!matrix(a[0], "logits", types[c], te[0], te[1], &l, &ldl) || !argument(a[1], "ids", types[I32], 2, choice, &ids, NULL) ||
        !argument(a[2], "probs", types[F32], 2, choice, &probs, NULL) || !where(a, names, 3, a[3], &st))
        return NULL;
    return PyLong_FromLong(block.route_fwd(l, ldl, (dlrm_dtype)c, (int)te[0], (int)te[1], (int)tk[1], ids, probs, st));
}

/* grad_probs, ids, probs, grad_logits, stream */
static PyObject* route_bwd(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    int64_t te[2], tk[2], ldl;
    void *gp, *ids, *probs, *l, *st;
    int c;
    static const char* const names[] = {"grad_probs", "ids", "probs", "grad_logits"};
    if (!ready(n, 5) || (c = type_code(a[3])) < 0 || !sizes(a[3], "grad_logits", 2, te) || !sizes(a[1], "ids", 2, tk))
        return NULL;
    const int64_t choice[2] = {te[0], tk[1]};
    if (!argument(a[0], "grad_probs", types[F32], 2, choice, &gp, NULL) ||
        !argument(a[1], "ids", types[I32], 2, choice, &ids, NULL) ||
        !argument(a[2], "probs", types[F32], 2, choice, &probs, NULL) ||
        !matrix(a[3], "grad_logits", types[c], te[0], te[1], &l, &ldl) || !where(a, names, 4, a[4], &st))
        return NULL;
    return PyLong_FromLong(block.route_bwd(gp, ids, probs, (dlrm_dtype)c, (int)te[0], (int)te[1], (int)tk[1], l, ldl, st));
}

/* ids, E, offsets, slots, order, workspace, status, stream */
static PyObject* expert_sort(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    int64_t tk[2];
    void *ids, *offsets, *slots, *order, *ws, *status, *st;
    size_t bytes;
    int E;
    static const char* const names[] = {"ids", NULL, "offsets", "slots", "order", "workspace", "status"};
    if (!ready(n, 8) || !sizes(a[0], "ids", 2, tk) || !code(a[1], "E", &E)) return NULL;
    if (!argument(a[0], "ids", types[I32], 2, tk, &ids, NULL) || !vector(a[2], "offsets", types[I32], (int64_t)E + 1, &offsets) ||
        !argument(a[3], "slots", types[I32], 2, tk, &slots, NULL) ||
        !vector(a[4], "order", types[I32], tk[0] * tk[1], &order) || !workspace(a[5], &ws, &bytes) ||
        !status_word(a[6], &status) || !where(a, names, 7, a[7], &st))
        return NULL;
    return PyLong_FromLong(block.expert_sort(ids, (int)tk[0], (int)tk[1], E, offsets, slots, order, ws, bytes, status, st));
}

/* x, slots, xs, status, stream */
static PyObject* dispatch_fwd(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    int64_t th[2], tk[2], rh[2], ldx, ldxs;
    void *x, *slots, *xs, *status, *st;
    int c;
    static const char* const names[] = {"x", "slots", "xs", "status"};
    if (!ready(n, 5) || (c = type_code(a[0])) < 0 || !sizes(a[0], "x", 2, th) || !sizes(a[1], "slots", 2, tk) ||
        !sizes(a[2], "xs", 2, rh))
        return NULL;
    const int64_t choice[2] = {th[0], tk[1]};
    if (!matrix(a[0], "x", types[c], th[0], th[1], &x, &ldx) || !argument(a[1], "slots", types[I32], 2, choice, &slots, NULL) ||
        !matrix(a[2], "xs", types[c], rh[0], th[1], &xs, &ldxs) || !status_word(a[3], &status) || !where(a, names, 4, a[4], &st))
        return NULL;
    return PyLong_FromLong(block.dispatch_fwd(x, ldx, slots, (dlrm_dtype)c, (int)th[0], (int)tk[1], (int)th[1], (int)rh[0], xs,
                                              ldxs, status, st));
}

/* grad_xs, slots, grad_x, status, stream */
static PyObject* dispatch_bwd(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    int64_t th[2], tk[2], rh[2], ldx, ldxs;
    void *x, *slots, *xs, *status, *st;
    int c;
    static const char* const names[] = {"grad_xs", "slots", "grad_x", "status"};
    if (!ready(n, 5) || (c = type_code(a[2])) < 0 || !sizes(a[2], "grad_x", 2, th) || !sizes(a[1], "slots", 2, tk) ||
        !sizes(a[0], "grad_xs", 2, rh))
        return NULL;
    const int64_t choice[2] = {th[0], tk[1]};
    if (!matrix(a[0], "grad_xs", types[c], rh[0], th[1], &xs, &ldxs) ||
        !argument(a[1], "slots", types[I32], 2, choice, &slots, NULL) ||
        !matrix(a[2], "grad_x", types[c], th[0], th[1], &x, &ldx) || !status_word(a[3], &status) ||
        !where(a, names, 4, a[4], &st))
        return NULL;
    return PyLong_FromLong(block.dispatch_bwd(xs, ldxs, slots, (dlrm_dtype)c, (int)th[0], (int)tk[1], (int)th[1], (int)rh[0], x,
                                              ldx, status, st));
}

/* ys, slots, probs, residual, y, status, stream */
static PyObject* combine_fwd(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    int64_t th[2], tk[2], rh[2], ldys, ldr, ldy;
    void *ys, *slots, *probs, *r, *y, *status, *st;
    int c;
    static const char* const names[] = {"ys", "slots", "probs", "residual", "y", "status"};
    if (!ready(n, 7) || (c = type_code(a[4])) < 0 || !sizes(a[4], "y", 2, th) || !sizes(a[1], "slots", 2, tk) ||
        !sizes(a[0], "ys", 2, rh))
        return NULL;
    const int64_t choice[2] = {th[0], tk[1]};
    if (!matrix(a[0], "ys", types[c], rh[0], th[1], &ys, &ldys) ||
        !argument(a[1], "slots", types[I32], 2, choice, &slots, NULL) ||
        !argument(a[2], "probs", types[F32], 2, choice, &probs, NULL) ||
        !matrix(a[3], "residual", types[c], th[0], th[1], &r, &ldr) || !matrix(a[4], "y", types[c], th[0], th[1], &y, &ldy) ||
        !status_word(a[5], &status) || !where(a, names, 6, a[6], &st))
        return NULL;
    return PyLong_FromLong(block.combine_fwd(ys, ldys, slots, probs, r, ldr, (dlrm_dtype)c, (int)th[0], (int)tk[1], (int)th[1],
                                             (int)rh[0], y, ldy, status, st));
}

/* grad_y, ys, slots, probs, grad_ys, grad_probs, status, stream */
static PyObject* combine_bwd(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    int64_t th[2], tk[2], rh[2] = {0, 0}, ldgy, ldys, ldgys;
    void *gy, *ys, *slots, *probs, *gys, *gp, *status, *st;
    int c;
    static const char* const names[] = {"grad_y", "ys", "slots", "probs", "grad_ys", "grad_probs", "status"};
    if (!ready(n, 8) || (c = type_code(a[0])) < 0 || !sizes(a[0], "grad_y", 2, th) || !sizes(a[2], "slots", 2, tk)) return NULL;
    PyObject* const rows[2] = {a[1], a[4]};
    PyObject* any = some(rows, 2, "ys and grad_ys");
    if (!any || !sizes(any, any == a[1] ? "ys" : "grad_ys", 2, rh)) return NULL;
    const int64_t choice[2] = {th[0], tk[1]};
    if (!matrix(a[0], "grad_y", types[c], th[0], th[1], &gy, &ldgy) || !matrix(a[1], "ys", types[c], rh[0], th[1], &ys, &ldys) ||
        !argument(a[2], "slots", types[I32], 2, choice, &slots, NULL) ||
        !argument(a[3], "probs", types[F32], 2, choice, &probs, NULL) ||
        !matrix(a[4], "grad_ys", types[c], rh[0], th[1], &gys, &ldgys) ||
        !argument(a[5], "grad_probs", types[F32], 2, choice, &gp, NULL) || !status_word(a[6], &status) ||
        !where(a, names, 7, a[7], &st))
        return NULL;
    return PyLong_FromLong(block.combine_bwd(gy, ldgy, ys, ldys, slots, probs, (dlrm_dtype)c, (int)th[0], (int)tk[1], (int)th[1],
                                             (int)rh[0], gys, ldgys, gp, status, st));
}

/* Bytes and exponents of a matrix in 8 bits. */
static int packed(PyObject* q, PyObject* exps, const char* name, const char* ename, int64_t rows, int64_t cols, void** p,
                  int64_t* ld, void** pe)
{
    const int64_t e[2] = {rows, (cols + 31) / 32};
    return matrix(q, name, types[U8], rows, cols, p, ld) && argument(exps, ename, types[U8], 2, e, pe, NULL);
}

/* x, q, exps, stream */
static PyObject* pack8(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    int64_t mn[2], ldx, ldq;
    void *x, *q, *e, *st;
    int c;
    static const char* const names[] = {"x", "q", "exps"};
    if (!ready(n, 4) || (c = type_code(a[0])) < 0 || !sizes(a[0], "x", 2, mn) ||
        !matrix(a[0], "x", types[c], mn[0], mn[1], &x, &ldx) || !packed(a[1], a[2], "q", "exps", mn[0], mn[1], &q, &ldq, &e) ||
        !where(a, names, 3, a[3], &st))
        return NULL;
    return PyLong_FromLong(block.pack8(x, ldx, (dlrm_dtype)c, (int)mn[0], (int)mn[1], q, ldq, e, st));
}

/* q, exps, y, stream */
static PyObject* unpack8(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    int64_t mn[2], ldy, ldq;
    void *y, *q, *e, *st;
    int c;
    static const char* const names[] = {"q", "exps", "y"};
    if (!ready(n, 4) || (c = type_code(a[2])) < 0 || !sizes(a[2], "y", 2, mn) ||
        !packed(a[0], a[1], "q", "exps", mn[0], mn[1], &q, &ldq, &e) || !matrix(a[2], "y", types[c], mn[0], mn[1], &y, &ldy) ||
        !where(a, names, 3, a[3], &st))
        return NULL;
    return PyLong_FromLong(block.unpack8(q, ldq, e, (dlrm_dtype)c, (int)mn[0], (int)mn[1], y, ldy, st));
}

/* grad_y, x_q, x_exps, w, pre_q, pre_exps, grad_x, grad_w, grad_bias, act, p, rng, workspace, status, stream */
static PyObject* linear_bwd8(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    int64_t mn[2], nk[2], ldg, ldx, ldw, ldp, lddx, lddw;
    void *g, *x, *xe, *w, *z, *ze, *dx, *dw, *db, *rng, *ws, *status, *st;
    size_t bytes;
    double p;
    int c, act;
    static const char* const names[] = {"grad_y", "x_q",    "x_exps",    "w",  "pre_q", "pre_exps", "grad_x",
                                        "grad_w", "grad_bias", NULL,     NULL, "rng",   "workspace", "status"};
    if (!ready(n, 15) || (c = type_code(a[0])) < 0 || !sizes(a[0], "grad_y", 2, mn) || !sizes(a[3], "w", 2, nk)) return NULL;
    PyObject* t = types[c];
    const int64_t M = mn[0], N = nk[0], K = nk[1];
    if (!matrix(a[0], "grad_y", t, M, N, &g, &ldg) || !packed(a[1], a[2], "x_q", "x_exps", M, K, &x, &ldx, &xe) ||
        !matrix(a[3], "w", t, N, K, &w, &ldw) || !packed(a[4], a[5], "pre_q", "pre_exps", M, N, &z, &ldp, &ze) ||
        !matrix(a[6], "grad_x", t, M, K, &dx, &lddx) || !matrix(a[7], "grad_w", t, N, K, &dw, &lddw) ||
        !vector(a[8], "grad_bias", types[F32], N, &db) || !code(a[9], "act", &act) || !real(a[10], &p) ||
        !vector(a[11], "rng", types[I64], 2, &rng) || !workspace(a[12], &ws, &bytes) || !status_word(a[13], &status) ||
        !where(a, names, 14, a[14], &st))
        return NULL;
    return PyLong_FromLong(block.linear_bwd8(g, ldg, x, ldx, xe, w, ldw, z, ldp, ze, (dlrm_dtype)c, (int)M, (int)N, (int)K,
                                             (dlrm_act)act, p, rng, dx, lddx, dw, lddw, db, ws, bytes, status, st));
}

/* bind_block(uint8 dtype, (addresses of the entry points in the order of `block`)), after bind */
static PyObject* bind_block(PyObject* self, PyObject* args)
{
    PyObject *u8, *at;
    if (!PyArg_ParseTuple(args, "OO!", &u8, &PyTuple_Type, &at) || !count(PyTuple_GET_SIZE(at), N_BLOCK)) return NULL;
    void* p[N_BLOCK];
    for (int i = 0; i < N_BLOCK; ++i) {
        p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(at, i));
        if (PyErr_Occurred()) return NULL;
    }
    Py_XSETREF(types[U8], Py_NewRef(u8));
    void** const to[N_BLOCK] = {(void**)&block.block_norm_fwd, (void**)&block.block_norm_bwd, (void**)&block.route_fwd,
                                (void**)&block.route_bwd,      (void**)&block.expert_sort,    (void**)&block.dispatch_fwd,
                                (void**)&block.dispatch_bwd,   (void**)&block.combine_fwd,    (void**)&block.combine_bwd,
                                (void**)&block.pack8,          (void**)&block.unpack8,        (void**)&block.linear_bwd8};
    for (int i = 0; i < N_BLOCK; ++i) *to[i] = p[i];
    Py_RETURN_NONE;
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
    {"bind_block", bind_block, METH_VARARGS, NULL},
#define BLOCK(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
    BLOCK(block_norm_fwd), BLOCK(block_norm_bwd), BLOCK(route_fwd), BLOCK(route_bwd), BLOCK(expert_sort), BLOCK(dispatch_fwd),
    BLOCK(dispatch_bwd), BLOCK(combine_fwd), BLOCK(combine_bwd), BLOCK(pack8), BLOCK(unpack8), BLOCK(linear_bwd8),
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
