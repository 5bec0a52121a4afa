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

typedef int (*route_fn)(const void *, int, int64_t, const float *, const uint8_t *, int64_t, int64_t,
                        int, int, int, int, int, int, float, int32_t *, float *, int32_t *,
                        int32_t *, int32_t *, void *, size_t, stream_t);
typedef size_t (*route_size_fn)(int64_t, int64_t, int);
typedef int (*group_fn)(const int32_t *, int64_t, int64_t, int32_t *, int32_t *, int32_t *, void *,
                        size_t, stream_t);
typedef size_t (*group_size_fn)(int64_t, int64_t);
typedef int (*combine_fn)(const void *, int, int64_t, int64_t, const int32_t *, const float *,
                          const void *, int64_t, void *, int, int64_t, int64_t, int64_t, int64_t,
                          stream_t);
typedef int (*adapter_fn)(const void *, int, int64_t, const void *, const void *, const int32_t *,
                          const int32_t *, const float *, const void *, int64_t, void *, int,
                          int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int, void *,
                          size_t, stream_t);
typedef size_t (*adapter_size_fn)(int64_t, int64_t, int64_t, int64_t, int);

static norm_fn f_norm;
static ragged_fn f_ragged;
static int8_fn f_int8;
static quant_fn f_quant;
static route_fn f_route;
static route_size_fn f_route_size;
static group_fn f_group;
static group_size_fn f_group_size;
static combine_fn f_combine;
static adapter_fn f_adapter;
static adapter_size_fn f_adapter_size;

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

/* ---- The calls on tensors.  sandwich_norm's checks read some thirty attributes, which
 * takes Python code 2 us, as long as the launch, and half as long here.  These entries
 * only take the plain case: every output given, every tensor dense.  Anything else,
 * what is to be refused included, is None: the Python code looks at it. */
enum { DIMS = 3 };
typedef struct {
    void *ptr;
    int64_t size[DIMS];
    int dims;
    PyObject *dtype;       /* borrowed: torch keeps its dtypes */
} tensor_t;

/* The attributes that are read: their names, and what a plain torch.Tensor's type has for
 * them (a subclass may have others), which saves the search for each. */
enum { SHAPE, DTYPE, DENSE, PTR_OF, BYTES, GPU_OF, ATTRS };
static const char *const attr_names[ATTRS] = {"shape", "dtype", "is_contiguous", "data_ptr",
                                              "element_size", "get_device"};
static PyObject *names[ATTRS], *own[ATTRS];
static PyTypeObject *plain;

static PyObject *get(PyObject *t, int a)
{
    if (Py_TYPE(t) == plain)
        return Py_TYPE(own[a])->tp_descr_get(own[a], t, (PyObject *)plain);
    return PyObject_GetAttr(t, names[a]);
}

static PyObject *call(PyObject *t, int a)
{
    if (Py_TYPE(t) == plain)
        return PyObject_Vectorcall(own[a], &t, 1, NULL);
    return PyObject_CallMethodNoArgs(t, names[a]);
}

/* Whether t is on the GPU *gpu (ANY_GPU: on any, which it becomes); an error may be set. */
enum { ANY_GPU = -1 };
static int on_gpu(PyObject *t, long *gpu)
{
    PyObject *o = call(t, GPU_OF);
    const long device = o ? PyLong_AsLong(o) : -1;       /* -1 for a tensor on no GPU */
    Py_XDECREF(o);
    if (device < 0 || (*gpu != ANY_GPU && device != *gpu))
        return 0;
    *gpu = device;
    return 1;
}

/* one_gpu(tensors ...): whether those that are not None are on one GPU */
static PyObject *py_one_gpu(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    (void)self;
    long gpu = ANY_GPU;
    int ok = names[0] != NULL;
    for (Py_ssize_t i = 0; ok && i < n; ++i)
        ok = args[i] == Py_None || on_gpu(args[i], &gpu);
    PyErr_Clear();
    return PyBool_FromLong(ok);
}

/* 1 for a dense tensor of one to three dimensions on the GPU *gpu (see on_gpu), else 0 (with
 * or without an error set). */
static int dense(PyObject *t, tensor_t *d, long *gpu)
{
    PyObject *o = get(t, SHAPE);
    int ok = o && PyTuple_Check(o) && PyTuple_GET_SIZE(o) >= 1 && PyTuple_GET_SIZE(o) <= DIMS;
    if (ok) {
        d->dims = (int)PyTuple_GET_SIZE(o);
        for (int i = 0; i < d->dims; ++i)
            d->size[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(o, i));
    }
    Py_XDECREF(o);
    if (!ok || !(o = get(t, DTYPE)))
        return 0;
    d->dtype = o;
    Py_DECREF(o);
    if (!on_gpu(t, gpu) || !(o = call(t, DENSE)))
        return 0;
    ok = o == Py_True;
    Py_DECREF(o);
    if (!ok || !(o = call(t, PTR_OF)))
        return 0;
    d->ptr = (void *)(uintptr_t)PyLong_AsUnsignedLongLong(o);
    Py_DECREF(o);
    return !PyErr_Occurred();
}

/* The stream argument: an address, or None for torch's current stream, by its functions
 * that bind_torch got.  Sets an error for anything else. */
static PyObject *current_raw, *current_device;
static void *stream_of(PyObject *s)
{
    if (s != Py_None)
        return PyLong_AsVoidPtr(s);
    PyObject *dev = current_device ? PyObject_CallNoArgs(current_device) : NULL;
    PyObject *raw = dev ? PyObject_CallOneArg(current_raw, dev) : NULL;
    void *p = raw ? PyLong_AsVoidPtr(raw) : NULL;
    if (!raw && !PyErr_Occurred())
        PyErr_SetString(PyExc_RuntimeError, "bind_torch() first");
    Py_XDECREF(dev);
    Py_XDECREF(raw);
    return p;
}

static int is(const tensor_t *d, int dims, int64_t a, int64_t b)
{
    return d->dims == dims && d->size[0] == a && (dims == 1 || d->size[1] == b);
}

/* torch's dtypes as the wrappers hand them over: int8, float32, then the output types in
 * the order of their codes. */
enum { T_INT8, T_F32, T_OUT };
static PyObject *type_at(PyObject *types, int i)
{
    return PyTuple_Check(types) && i >= 0 && i < PyTuple_GET_SIZE(types) ? PyTuple_GET_ITEM(types, i) : NULL;
}

/* h, x, w_post, w_pre, gate, gate_rows, res_scale, eps, kind, x_out, y_out, scales_out,
 * the input types' codes by dtype, dtypes, stream */
static PyObject *py_norm_tensors(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    (void)self;
    if (!want(n, 15, f_norm != NULL))
        return NULL;
    tensor_t h, x, xo, y, t;
    void *post = NULL, *pre = NULL, *gate = NULL, *scales = NULL;
    int64_t gate_rows = 1, M, D;
    long gpu = ANY_GPU;
    const int kind = I32(8);
    if (!dense(args[0], &h, &gpu) || h.dims != 2 || !dense(args[1], &x, &gpu) || !dense(args[9], &xo, &gpu) ||
        !dense(args[10], &y, &gpu))
        goto other;
    M = h.size[0], D = h.size[1];
    if (!is(&x, 2, M, D) || !is(&xo, 2, M, D) || !is(&y, 2, M, D) || xo.dtype != x.dtype ||
        (kind == 0 && y.dtype != h.dtype))
        goto other;
    if (kind != 0) {
        PyObject *o = call(args[10], BYTES);
        const long bytes = o ? PyLong_AsLong(o) : 0;
        Py_XDECREF(o);
        if (bytes != 1 || !dense(args[11], &t, &gpu) || t.dtype != type_at(args[13], T_F32) ||
            !(kind == 1 ? is(&t, 2, M, (D + 127) / 128) : is(&t, 1, M, 0)))
            goto other;
        scales = t.ptr;
    }
    if (args[2] != Py_None) {
        if (!dense(args[2], &t, &gpu) || !is(&t, 1, D, 0) || t.dtype != h.dtype)
            goto other;
        post = t.ptr;
    }
    if (args[3] != Py_None) {
        if (!dense(args[3], &t, &gpu) || !is(&t, 1, D, 0) || t.dtype != h.dtype)
            goto other;
        pre = t.ptr;
    }
    if (args[4] != Py_None) {
        if (!dense(args[4], &t, &gpu) || t.dims > 2 || t.size[t.dims - 1] != D || t.dtype != h.dtype)
            goto other;
        const int64_t rows = t.dims == 2 ? t.size[0] : 1;
        if (args[5] != Py_None)
            gate_rows = I64(5);
        else if (rows > 0)
            gate_rows = (M + rows - 1) / rows > 1 ? (M + rows - 1) / rows : 1;
        if (gate_rows < 1 || rows < (M + gate_rows - 1) / gate_rows)
            goto other;
        gate = t.ptr;
    }
    PyObject *hk = PyDict_GetItemWithError(args[12], h.dtype);
    PyObject *xk = PyDict_GetItemWithError(args[12], x.dtype);
    if (!hk || !xk)
        goto other;
    const int h_code = (int)PyLong_AsLong(hk), x_code = (int)PyLong_AsLong(xk);
    const double rs = PyFloat_AsDouble(args[6]), eps = PyFloat_AsDouble(args[7]);
    void *s = stream_of(args[14]);
    if (PyErr_Occurred())
        goto other;
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = f_norm(h.ptr, h_code, 0, x.ptr, x_code, 0, post, gate, gate_rows, pre, (float)rs, (float)eps,
                xo.ptr, 0, y.ptr, scales, kind, 0, M, D, s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
other:
    PyErr_Clear();
    Py_RETURN_NONE;
}

/* A, a_s, B, b_s, out, output code, dtypes, stream */
static PyObject *py_int8_tensors(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    (void)self;
    if (!want(n, 8, f_int8 != NULL))
        return NULL;
    tensor_t a, as, b, bs, c;
    int st;
    long gpu = ANY_GPU;
    const int out = I32(5);
    PyObject *const i8 = type_at(args[6], T_INT8), *const f32 = type_at(args[6], T_F32);
    if (dense(args[0], &a, &gpu) && dense(args[1], &as, &gpu) && dense(args[2], &b, &gpu) && dense(args[3], &bs, &gpu) &&
        dense(args[4], &c, &gpu) && a.dtype == i8 && b.dtype == i8 && as.dtype == f32 && bs.dtype == f32 &&
        out >= 0 && c.dtype == type_at(args[6], T_OUT + out) && a.dims == 2 && b.dims == 2 &&
        a.size[1] == b.size[1] && is(&as, 1, a.size[0], 0) && is(&bs, 1, b.size[0], 0) &&
        is(&c, 2, a.size[0], b.size[0])) {
        void *s = stream_of(args[7]);
        if (!PyErr_Occurred()) {
            Py_BEGIN_ALLOW_THREADS
            st = f_int8(a.ptr, 0, as.ptr, b.ptr, 0, bs.ptr, c.ptr, 0, a.size[0], b.size[0], a.size[1], out,
                        s, NULL);
            Py_END_ALLOW_THREADS
            return PyLong_FromLong(st);
        }
    }
    PyErr_Clear();
    Py_RETURN_NONE;
}

/* X, A, a_s, the input types' codes by dtype, dtypes, stream */
static PyObject *py_quant_tensors(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    (void)self;
    if (!want(n, 6, f_quant != NULL))
        return NULL;
    tensor_t x, a, as;
    int st;
    long gpu = ANY_GPU;
    if (dense(args[0], &x, &gpu) && dense(args[1], &a, &gpu) && dense(args[2], &as, &gpu) && x.dims == 2 &&
        a.dtype == type_at(args[4], T_INT8) && as.dtype == type_at(args[4], T_F32) &&
        is(&a, 2, x.size[0], x.size[1]) && is(&as, 1, x.size[0], 0)) {
        PyObject *code = PyDict_GetItemWithError(args[3], x.dtype);
        const int kind = code ? (int)PyLong_AsLong(code) : -1;
        void *s = stream_of(args[5]);
        if (code && !PyErr_Occurred()) {
            Py_BEGIN_ALLOW_THREADS
            st = f_quant(x.ptr, kind, 0, a.ptr, 0, as.ptr, x.size[0], x.size[1], s);
            Py_END_ALLOW_THREADS
            return PyLong_FromLong(st);
        }
    }
    PyErr_Clear();
    Py_RETURN_NONE;
}

static int is3(const tensor_t *d, int64_t a, int64_t b, int64_t c)
{
    return d->dims == 3 && d->size[0] == a && d->size[1] == b && d->size[2] == c;
}

/* Whether the GPU is the current one, by torch's function that bind_torch got. */
static int is_current(long gpu)
{
    PyObject *o = current_device ? PyObject_CallNoArgs(current_device) : NULL;
    const int ok = o && PyLong_AsLong(o) == gpu;
    Py_XDECREF(o);
    return ok;
}

/* A new tensor [a], or with b >= 0 [a, b], of dtype on t's device and the current stream; a
 * new reference and its address, or NULL with an error set.  (Between launches a tensor
 * costs some 2.5 us on the host, by this or another of torch's calls: loops give outputs.) */
static PyObject *new_tensor(PyObject *t, int64_t a, int64_t b, PyObject *dtype, void **ptr)
{
    static PyObject *new_empty, *kw;
    if (!new_empty && !(new_empty = PyUnicode_InternFromString("new_empty")))
        return NULL;
    if (!kw && !(kw = Py_BuildValue("(s)", "dtype")))
        return NULL;
    PyObject *call_args[4] = {t, PyLong_FromLongLong(a)};
    int n = 2;
    if (b >= 0)
        call_args[n++] = PyLong_FromLongLong(b);
    call_args[n] = dtype;
    PyObject *made = NULL;
    if (call_args[1] && call_args[n - 1])
        made = PyObject_VectorcallMethod(new_empty, call_args, n, kw);
    for (int i = 1; i < n; ++i)
        Py_XDECREF(call_args[i]);
    PyObject *o = made ? call(made, PTR_OF) : NULL;
    if (o)
        *ptr = (void *)(uintptr_t)PyLong_AsUnsignedLongLong(o);
    Py_XDECREF(o);
    if (o && !PyErr_Occurred())
        return made;
    Py_XDECREF(made);
    return NULL;
}

/* Device scratch of `bytes`: NULL and no address for 0.  0 on an error. */
static int scratch_of(PyObject *t, size_t bytes, PyObject *u8, PyObject **keep, void **ptr)
{
    *keep = NULL;
    *ptr = NULL;
    return !bytes || (u8 && (*keep = new_tensor(t, (int64_t)bytes, -1, u8, ptr)) != NULL);
}

/* The types of the routing calls: int32, float32, bool, uint8. */
enum { R_INT32, R_F32, R_BOOL, R_U8 };

/* A dense tensor of `dims` dimensions and of that type */
static int typed(PyObject *o, tensor_t *t, long *gpu, int dims, PyObject *dtype)
{
    return dtype && dense(o, t, gpu) && t->dims == dims && t->dtype == dtype;
}

/* What a call returns that made its outputs (takes the reference), or was given them (NULL). */
static PyObject *result_of(PyObject *made, int st)
{
    if (made && !st)
        return made;
    Py_XDECREF(made);
    return PyLong_FromLong(st);
}

static int code_of(PyObject *codes, PyObject *dtype)
{
    PyObject *o = PyDict_GetItemWithError(codes, dtype);
    return o ? (int)PyLong_AsLong(o) : -1;
}

/* Whether a positive number stays what it is in the C call's 32 bits. */
static int fits32(int64_t v) { return v >= 1 && v <= INT32_MAX; }

/* logits, top_k, scoring, bias, groups, top_groups, group_top, renormalize, scale, valid,
 * outputs, the input types' codes by dtype, dtypes, stream.  Without outputs (None), here and
 * below, the result is a tuple of new ones (one: the tensor), or a status other than 0. */
static PyObject *py_route_tensors(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    (void)self;
    if (!want(n, 14, f_route != NULL))
        return NULL;
    tensor_t x, bias = {0}, valid = {0}, o[5];
    long gpu = ANY_GPU;
    const int make = args[10] == Py_None;
    PyObject *made = NULL, *keep = NULL;
    PyObject *const i32 = type_at(args[12], R_INT32), *const f32 = type_at(args[12], R_F32);
    if ((!make && (!PyTuple_Check(args[10]) || PyTuple_GET_SIZE(args[10]) != 5)) || !PyLong_Check(args[1]) ||
        !dense(args[0], &x, &gpu) || x.dims != 2)
        goto other;
    const int64_t T = x.size[0], E = x.size[1], k = I64(1);
    if (k < 1 || k > 32)
        goto other;
    if (args[3] != Py_None && (!typed(args[3], &bias, &gpu, 1, f32) || !is(&bias, 1, E, 0)))
        goto other;
    if (args[9] != Py_None && (!dense(args[9], &valid, &gpu) || !is(&valid, 1, T, 0) ||
                               (valid.dtype != type_at(args[12], R_BOOL) && valid.dtype != type_at(args[12], R_U8))))
        goto other;
    for (int i = 0; i < 5 && !make; ++i) {
        const int flat = i == 2 || i == 3;
        if (!typed(PyTuple_GET_ITEM(args[10], i), &o[i], &gpu, flat ? 1 : 2, i == 1 ? f32 : i32) ||
            !(flat ? is(&o[i], 1, i == 2 ? T * k : E + 1, 0) : is(&o[i], 2, T, k)))
            goto other;
    }
    const int kind = code_of(args[11], x.dtype), renormalize = PyObject_IsTrue(args[7]);
    const double scale = PyFloat_AsDouble(args[8]);
    const int64_t groups = I64(4), top_groups = I64(5), group_top = I64(6);
    const int scoring = I32(2);
    const size_t size = f_route_size(T, E, (int)k);
    if (!fits32(groups) || !fits32(top_groups) || !fits32(group_top) || kind < 0 || renormalize < 0 || !is_current(gpu) || ((size || make) && args[13] != Py_None) ||
        PyErr_Occurred())
        goto other;
    if (make) {
        if (!i32 || !f32 || !(made = PyTuple_New(5)))
            goto other;
        for (int i = 0; i < 5; ++i) {
            const int flat = i == 2 || i == 3;
            PyObject *const t = new_tensor(args[0], !flat ? T : i == 2 ? T * k : E + 1, flat ? -1 : k,
                                           i == 1 ? f32 : i32, &o[i].ptr);
            if (!t)
                goto other;
            PyTuple_SET_ITEM(made, i, t);
        }
    }
    void *s = stream_of(args[13]), *scratch;
    if (PyErr_Occurred() || !scratch_of(args[0], size, type_at(args[12], R_U8), &keep, &scratch))
        goto other;
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = f_route(x.ptr, kind, 0, bias.ptr, valid.ptr, T, E, (int)k, scoring, (int)groups, (int)top_groups,
                 (int)group_top, renormalize, (float)scale, o[0].ptr, o[1].ptr, o[2].ptr, o[3].ptr, o[4].ptr, scratch, size, s);
    Py_END_ALLOW_THREADS
    Py_XDECREF(keep);
    return result_of(made, st);
other:
    PyErr_Clear();
    Py_XDECREF(made);
    Py_RETURN_NONE;
}

/* ids, groups, outputs, dtypes, stream */
static PyObject *py_group_tensors(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    (void)self;
    if (!want(n, 5, f_group != NULL))
        return NULL;
    tensor_t ids, order, offsets;
    PyObject *made[2] = {NULL, NULL}, *keep = NULL;
    long gpu = ANY_GPU;
    PyObject *const i32 = type_at(args[3], R_INT32);
    if (!PyLong_Check(args[1]) || !typed(args[0], &ids, &gpu, 1, i32))
        goto other;
    const int64_t count = ids.size[0], groups = I64(1);
    if (groups < 1 || groups > 1024 || !is_current(gpu))
        goto other;
    const size_t size = f_group_size(count, groups);
    if ((size || args[2] == Py_None) && args[4] != Py_None)
        goto other;
    if (args[2] == Py_None) {
        if (!(made[0] = new_tensor(args[0], count, -1, i32, &order.ptr)) ||
            !(made[1] = new_tensor(args[0], groups + 1, -1, i32, &offsets.ptr)))
            goto other;
    } else if (!PyTuple_Check(args[2]) || PyTuple_GET_SIZE(args[2]) != 2 ||
               !typed(PyTuple_GET_ITEM(args[2], 0), &order, &gpu, 1, i32) || !is(&order, 1, count, 0) ||
               !typed(PyTuple_GET_ITEM(args[2], 1), &offsets, &gpu, 1, i32) || !is(&offsets, 1, groups + 1, 0)) {
        goto other;
    }
    void *s = stream_of(args[4]), *scratch;
    if (PyErr_Occurred() || !scratch_of(args[0], size, type_at(args[3], R_U8), &keep, &scratch))
        goto other;
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = f_group(ids.ptr, count, groups, order.ptr, offsets.ptr, NULL, scratch, size, s);
    Py_END_ALLOW_THREADS
    PyObject *result = made[0] && !st ? PyTuple_Pack(2, made[0], made[1]) : PyLong_FromLong(st);
    Py_XDECREF(keep);
    Py_XDECREF(made[0]);
    Py_XDECREF(made[1]);
    return result;
other:
    PyErr_Clear();
    Py_XDECREF(made[0]);
    Py_XDECREF(made[1]);
    Py_RETURN_NONE;
}

/* Y, rows, weights, add, out (or a new one's dtype, None: Y's), the input types' codes by dtype,
 * dtypes, stream */
static PyObject *py_combine_tensors(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    (void)self;
    if (!want(n, 8, f_combine != NULL))
        return NULL;
    tensor_t y, rows, weights, add = {0}, out;
    long gpu = ANY_GPU;
    const int make = Py_TYPE(args[4]) != plain;
    PyObject *made = NULL;
    if (!dense(args[0], &y, &gpu) || y.dims != 2 || !typed(args[1], &rows, &gpu, 2, type_at(args[6], R_INT32)) ||
        !typed(args[2], &weights, &gpu, 2, type_at(args[6], R_F32)) ||
        !is(&weights, 2, rows.size[0], rows.size[1]))
        goto other;
    if (make) {
        if (args[7] != Py_None || !is_current(gpu) || (args[4] != Py_None && code_of(args[5], args[4]) < 0))
            goto other;
        out.dtype = args[4] == Py_None ? y.dtype : args[4];
        out.dims = 2;
        out.size[0] = rows.size[0];
        out.size[1] = y.size[1];
    } else if (!dense(args[4], &out, &gpu) || !is(&out, 2, rows.size[0], y.size[1])) {
        goto other;
    }
    if (args[3] != Py_None && (!typed(args[3], &add, &gpu, 2, out.dtype) || !is(&add, 2, out.size[0], out.size[1])))
        goto other;
    const int y_kind = code_of(args[5], y.dtype), out_kind = code_of(args[5], out.dtype);
    if (y_kind < 0 || out_kind < 0 || !is_current(gpu))
        goto other;
    if (make && !(made = new_tensor(args[0], out.size[0], out.size[1], out.dtype, &out.ptr)))
        goto other;
    void *s = stream_of(args[7]);
    if (PyErr_Occurred())
        goto other;
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = f_combine(y.ptr, y_kind, 0, y.size[0], rows.ptr, weights.ptr, add.ptr, 0, out.ptr, out_kind, 0,
                   rows.size[0], rows.size[1], y.size[1], s);
    Py_END_ALLOW_THREADS
    return result_of(made, st);
other:
    PyErr_Clear();
    Py_XDECREF(made);
    Py_RETURN_NONE;
}

/* x, A, B, order, offsets, base, scales, out, the input types' codes by dtype, dtypes, stream */
static PyObject *py_adapter_tensors(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    (void)self;
    if (!want(n, 11, f_adapter != NULL))
        return NULL;
    tensor_t x, a, b, order, offsets, base, scales = {0}, out;
    long gpu = ANY_GPU;
    const int make = args[7] == Py_None;
    PyObject *made = NULL, *keep = NULL;
    PyObject *const i32 = type_at(args[9], R_INT32);
    if (!dense(args[0], &x, &gpu) || x.dims != 2 || !typed(args[1], &a, &gpu, 3, x.dtype) ||
        !typed(args[2], &b, &gpu, 3, x.dtype) || !typed(args[3], &order, &gpu, 1, i32) ||
        !typed(args[4], &offsets, &gpu, 1, i32) || !dense(args[5], &base, &gpu) ||
        (!make && !dense(args[7], &out, &gpu)))
        goto other;
    const int64_t T = x.size[0], K = x.size[1], L = a.size[0], r = a.size[1], N = b.size[1];
    if (!is3(&a, L, r, K) || !is3(&b, L, N, r) || !is(&order, 1, T, 0) || !is(&offsets, 1, L + 1, 0) ||
        !is(&base, 2, T, N) || (!make && (!is(&out, 2, T, N) || out.dtype != base.dtype)))
        goto other;
    if (args[6] != Py_None && (!typed(args[6], &scales, &gpu, 1, type_at(args[9], R_F32)) || !is(&scales, 1, L, 0)))
        goto other;
    const int kind = code_of(args[8], x.dtype), out_kind = code_of(args[8], base.dtype);
    const size_t size = f_adapter_size(T, L, r, K, 0);
    if (kind < 0 || out_kind < 0 || !is_current(gpu) || ((size || make) && args[10] != Py_None))
        goto other;
    if (make && !(made = new_tensor(args[5], T, N, base.dtype, &out.ptr)))
        goto other;
    void *s = stream_of(args[10]), *scratch;
    if (PyErr_Occurred() || !scratch_of(args[0], size, type_at(args[9], R_U8), &keep, &scratch))
        goto other;
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = f_adapter(x.ptr, kind, 0, a.ptr, b.ptr, order.ptr, offsets.ptr, scales.ptr, base.ptr, 0, out.ptr, out_kind, 0,
                   T, L, r, K, N, 0, scratch, size, s);
    Py_END_ALLOW_THREADS
    Py_XDECREF(keep);
    return result_of(made, st);
other:
    PyErr_Clear();
    Py_XDECREF(made);
    Py_RETURN_NONE;
}

/* bind_routing(route, its workspace size, group, its workspace size, combine, adapter, its
 * workspace size) */
static PyObject *py_bind_routing(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    (void)self;
    if (!want(n, 7, 1))
        return NULL;
    f_route = (route_fn)PTR(0);
    f_route_size = (route_size_fn)PTR(1);
    f_group = (group_fn)PTR(2);
    f_group_size = (group_size_fn)PTR(3);
    f_combine = (combine_fn)PTR(4);
    f_adapter = (adapter_fn)PTR(5);
    f_adapter_size = (adapter_size_fn)PTR(6);
    if (PyErr_Occurred())
        return NULL;
    Py_RETURN_NONE;
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
    for (int i = 0; i < ATTRS && !names[i]; ++i)
        names[i] = PyUnicode_InternFromString(attr_names[i]);
    if (PyErr_Occurred())
        return NULL;
    Py_RETURN_NONE;
}

/* bind_torch(torch.Tensor, current raw stream of a device, current device) */
static PyObject *py_bind_torch(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    (void)self;
    if (!want(n, 3, names[0] != NULL))
        return NULL;
    if (plain)                       /* torch does not change */
        Py_RETURN_NONE;
    for (int i = 0; i < ATTRS; ++i) {
        if (!(own[i] = PyObject_GetAttr(args[0], names[i])))
            return NULL;
        if ((i == SHAPE || i == DTYPE) && !Py_TYPE(own[i])->tp_descr_get) {
            PyErr_SetString(PyExc_TypeError, "torch.Tensor: shape and dtype are no descriptors");
            return NULL;
        }
    }
    current_raw = Py_NewRef(args[1]);
    current_device = Py_NewRef(args[2]);
    plain = (PyTypeObject *)Py_NewRef(args[0]);
    Py_RETURN_NONE;
}

#define ENTRY(name, fn, doc) {name, (PyCFunction)(void (*)(void))fn, METH_FASTCALL, doc}
static PyMethodDef methods[] = {
    ENTRY("bind", py_bind, "set the library's function addresses"),
    ENTRY("bind_torch", py_bind_torch, "torch's tensor type, and its functions for the current stream"),
    ENTRY("bind_routing", py_bind_routing, "set the addresses of the routing calls"),
    ENTRY("route_tensors", py_route_tensors, "route_experts, as norm_tensors"),
    ENTRY("group_tensors", py_group_tensors, "group_rows, as norm_tensors"),
    ENTRY("combine_tensors", py_combine_tensors, "combine_experts, as norm_tensors"),
    ENTRY("adapter_tensors", py_adapter_tensors, "adapter_matmul, as norm_tensors"),
    ENTRY("one_gpu", py_one_gpu, "whether tensors are on one GPU"),
    ENTRY("w8a8_sandwich_norm", py_norm, "see the C header"),
    ENTRY("norm_tensors", py_norm_tensors, "sandwich_norm of dense tensors with every output given"),
    ENTRY("int8_tensors", py_int8_tensors, "int8_matmul, as norm_tensors"),
    ENTRY("quant_tensors", py_quant_tensors, "quantize_int8_per_token, as norm_tensors"),
    ENTRY("w8a8_block_fp8_grouped_matmul_ragged", py_ragged, "see the C header"),
    ENTRY("w8a8_int8_matmul", py_int8, "see the C header"),
    ENTRY("w8a8_quantize_int8_per_token", py_quant, "see the C header"),
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_w8a8_pycall", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};
PyMODINIT_FUNC PyInit__w8a8_pycall(void) { return PyModule_Create(&module); }
