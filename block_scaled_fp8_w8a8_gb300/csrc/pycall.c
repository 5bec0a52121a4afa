/* Python entries of the calls that stand before kernels of a few microseconds:
 * the same arguments as the C functions (addresses and numbers as Python numbers,
 * None for a null pointer), converted without ctypes, which takes 1.9 us for the
 * 21 arguments of w8a8_sandwich_norm against 0.3 us here.  The functions'
 * addresses come from the loaded library (bind), so this module links to nothing.
 * The GIL is released during a call, as ctypes does. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

typedef struct CUstream_st *stream_t;
typedef int (*norm_fn)(const void *, int, int64_t, const void *, int, int64_t, const void *,
                       const void *, int64_t, const void *, float, float, void *, int64_t, void *,
                       float *, int, int64_t, int64_t, int64_t, stream_t);
typedef int (*ragged_fn)(const void *, const float *, const void *, const float *, void *,
                         const int32_t *, int64_t, int64_t, int64_t, int64_t, int, int, int,
                         stream_t, const void *);
typedef int (*int8_fn)(const void *, int64_t, const float *, const void *, int64_t, const float *,
                       void *, int64_t, int64_t, int64_t, int64_t, int, stream_t, const void *);
typedef int (*quant_fn)(const void *, int, int64_t, void *, int64_t, float *, int64_t, int64_t,
                        stream_t);

static norm_fn f_norm;
static ragged_fn f_ragged;
static int8_fn f_int8;
static quant_fn f_quant;

/* Argument i as an integer; None is 0.  Sets an error for anything else. */
static int64_t num(PyObject *const *args, int i)
{
    if (args[i] == Py_None)
        return 0;
    const int64_t v = PyLong_AsLongLong(args[i]);
    if (v == -1 && PyErr_Occurred()) {
        /* an address with the top bit set */
        PyErr_Clear();
        return (int64_t)PyLong_AsUnsignedLongLong(args[i]);
    }
    return v;
}
#define PTR(i) ((void *)(uintptr_t)num(args, i))
#define I64(i) num(args, i)
#define I32(i) ((int)num(args, i))

static int want(Py_ssize_t have, Py_ssize_t need, int bound)
{
    if (!bound)
        PyErr_SetString(PyExc_RuntimeError, "bind() first");
    else if (have != need)
        PyErr_Format(PyExc_TypeError, "%zd arguments, want %zd", have, need);
    else
        return 1;
    return 0;
}

static PyObject *py_norm(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    (void)self;
    if (!want(n, 21, f_norm != NULL))
        return NULL;
    void *h = PTR(0), *x = PTR(3), *wp = PTR(6), *gate = PTR(7), *wq = PTR(9), *xo = PTR(12),
         *y = PTR(14), *sc = PTR(15), *s = PTR(20);
    const int hk = I32(1), xk = I32(4), kind = I32(16);
    const int64_t lh = I64(2), lx = I64(5), gr = I64(8), lo = I64(13), ly = I64(17), M = I64(18),
                  D = I64(19);
    const double rs = PyFloat_AsDouble(args[10]), eps = PyFloat_AsDouble(args[11]);
    int st;
    if (PyErr_Occurred())
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = f_norm(h, hk, lh, x, xk, lx, wp, gate, gr, wq, (float)rs, (float)eps, xo, lo, y, sc, kind, ly,
                M, D, s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

static PyObject *py_ragged(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    (void)self;
    if (!want(n, 15, f_ragged != NULL))
        return NULL;
    void *A = PTR(0), *as = PTR(1), *B = PTR(2), *bs = PTR(3), *C = PTR(4), *off = PTR(5),
         *s = PTR(13), *o = PTR(14);
    const int64_t M = I64(6), E = I64(7), N = I64(8), K = I64(9);
    const int bn = I32(10), bk = I32(11), out = I32(12);
    int st;
    if (PyErr_Occurred())
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = f_ragged(A, as, B, bs, C, off, M, E, N, K, bn, bk, out, s, o);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

static PyObject *py_int8(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    (void)self;
    if (!want(n, 14, f_int8 != NULL))
        return NULL;
    void *A = PTR(0), *as = PTR(2), *B = PTR(3), *bs = PTR(5), *C = PTR(6), *s = PTR(12), *o = PTR(13);
    const int64_t la = I64(1), lb = I64(4), lc = I64(7), M = I64(8), N = I64(9), K = I64(10);
    const int out = I32(11);
    int st;
    if (PyErr_Occurred())
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = f_int8(A, la, as, B, lb, bs, C, lc, M, N, K, out, s, o);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

static PyObject *py_quant(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    (void)self;
    if (!want(n, 9, f_quant != NULL))
        return NULL;
    void *X = PTR(0), *A = PTR(3), *as = PTR(5), *s = PTR(8);
    const int kind = I32(1);
    const int64_t lx = I64(2), la = I64(4), M = I64(6), K = I64(7);
    int st;
    if (PyErr_Occurred())
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = f_quant(X, kind, lx, A, la, as, M, K, s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* bind(norm, ragged, int8, quant): addresses in the loaded library */
static PyObject *py_bind(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    (void)self;
    if (!want(n, 4, 1))
        return NULL;
    f_norm = (norm_fn)PTR(0);
    f_ragged = (ragged_fn)PTR(1);
    f_int8 = (int8_fn)PTR(2);
    f_quant = (quant_fn)PTR(3);
    if (PyErr_Occurred())
        return NULL;
    Py_RETURN_NONE;
}

#define ENTRY(name, fn, doc) {name, (PyCFunction)(void (*)(void))fn, METH_FASTCALL, doc}
static PyMethodDef methods[] = {
    ENTRY("bind", py_bind, "set the library's function addresses"),
    ENTRY("w8a8_sandwich_norm", py_norm, "see the C header"),
    ENTRY("w8a8_block_fp8_grouped_matmul_ragged", py_ragged, "see the C header"),
    ENTRY("w8a8_int8_matmul", py_int8, "see the C header"),
    ENTRY("w8a8_quantize_int8_per_token", py_quant, "see the C header"),
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_w8a8_pycall", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};
PyMODINIT_FUNC PyInit__w8a8_pycall(void) { return PyModule_Create(&module); }
