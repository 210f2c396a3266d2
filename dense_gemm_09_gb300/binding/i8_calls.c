/*
 * i8_calls.c -- CPython module _i8_calls: argument marshalling of the 8-bit
 * calls and the calls on tokens by expert, in C.
 *
 * These calls take a few microseconds of GPU time for one token, and through
 * ctypes a call spent 5 to 7 us on the host, most of it on reading and checking
 * tensors' attributes in Python; here it spends 3.5 to 4.6, of which the launch
 * itself is ~2.  The module does what the ctypes binding does for the other
 * calls: reads pointers, pitches and the current stream, checks shapes, types
 * and devices, calls the C ABI and raises.  It links neither torch nor the library:
 * tensors are read through their Python attributes, and the entry points'
 * addresses come with each call.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>

/* ---- what setup() hands over, and interned attribute names */

enum { F32 = 0, F16 = 1, BF16 = 2, I8 = 3, E4M3 = 4, E5M2 = 5, I32 = 6, I64 = 7, kTypes = 8 }; /* 0..2: dgemm_type */
static PyObject *g_dtype[kTypes];
static PyObject *g_get_device, *g_raw_stream, *g_error;
static PyObject *s_shape, *s_stride, *s_dtype, *s_is_cuda, *s_get_device, *s_data_ptr, *s_cuda_stream;

static PyObject *setup(PyObject *self, PyObject *args)
{
    PyObject *d[kTypes] = {NULL}, *dev, *raw, *err;
    (void)self;
    if (!PyArg_ParseTuple(args, "OOOOOOO|OOOO", &d[0], &d[1], &d[2], &d[3], &dev, &raw, &err, &d[4], &d[5], &d[6], &d[7]))
        return NULL;
    for (int i = 0; i < kTypes; ++i) {
        if (!d[i]) continue; /* as it was */
        Py_INCREF(d[i]);
        Py_XSETREF(g_dtype[i], d[i]);
    }
    Py_INCREF(dev);
    Py_XSETREF(g_get_device, dev);
    Py_INCREF(raw);
    Py_XSETREF(g_raw_stream, raw);
    Py_INCREF(err);
    Py_XSETREF(g_error, err);
    Py_RETURN_NONE;
}

/* ---- tensors */

typedef struct {
    void *ptr;
    int64_t ld;
    int64_t rows, cols;
    int type; /* index in g_dtype, -1 for any other */
} Mat;

static int type_of(PyObject *t)
{
    PyObject *d = PyObject_GetAttr(t, s_dtype);
    if (!d) {
        PyErr_Clear();
        return -1;
    }
    int code = -1;
    for (int i = 0; i < kTypes; ++i)
        if (d == g_dtype[i]) code = i;
    Py_DECREF(d);
    return code;
}

static int wrong_type(PyObject *t, const char *name, int want)
{
    PyObject *d = PyObject_GetAttr(t, s_dtype);
    if (!d) PyErr_Clear();
    PyErr_Format(PyExc_TypeError, "%s must be %S, got %S", name, g_dtype[want], d ? d : Py_None);
    Py_XDECREF(d);
    return -1;
}

/* Whether t is on the GPU of the call's tensors before it (*device; -1: none so
 * far).  The kernels run on one GPU, where another's addresses mean nothing. */
static int same_device(PyObject *t, const char *name, int64_t *device)
{
    PyObject *d = PyObject_CallMethodNoArgs(t, s_get_device);
    if (!d) return -1;
    const int64_t on = PyLong_AsLongLong(d);
    Py_DECREF(d);
    if (on == -1 && PyErr_Occurred()) return -1;
    if (*device < 0) *device = on;
    if (on == *device) return 0;
    PyErr_Format(PyExc_ValueError, "%s is on cuda:%lld, another tensor of the call on cuda:%lld", name, (long long)on,
                 (long long)*device);
    return -1;
}

static int on_gpu(PyObject *t)
{
    PyObject *c = PyObject_GetAttr(t, s_is_cuda);
    if (!c) {
        PyErr_Clear();
        return 0;
    }
    const int yes = c == Py_True;
    Py_DECREF(c);
    return yes;
}

/* n integers of a tuple; 0 on success, -1 without an exception set otherwise */
static int ints(PyObject *tuple, Py_ssize_t n, int64_t *out)
{
    if (!tuple || !PyTuple_Check(tuple) || PyTuple_GET_SIZE(tuple) != n) return -1;
    for (Py_ssize_t i = 0; i < n; ++i) {
        out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
        if (out[i] == -1 && PyErr_Occurred()) return -1;
    }
    return 0;
}

/* shape and strides of an n-dimensional tensor */
static int layout(PyObject *t, Py_ssize_t n, int64_t *shape, int64_t *stride)
{
    PyObject *a = PyObject_GetAttr(t, s_shape);
    int st = ints(a, n, shape);
    Py_XDECREF(a);
    if (st == 0) {
        a = PyObject_CallMethodNoArgs(t, s_stride);
        st = ints(a, n, stride);
        Py_XDECREF(a);
    }
    if (st != 0) PyErr_Clear();
    return st;
}

static int address(PyObject *t, void **ptr)
{
    PyObject *p = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!p) return -1;
    *ptr = PyLong_AsVoidPtr(p);
    Py_DECREF(p);
    return *ptr == NULL && PyErr_Occurred() ? -1 : 0;
}

/* A matrix of type `want`, or with want < 0 of any float type. */
static int matrix(PyObject *t, const char *name, int want, Mat *m, int64_t *device)
{
    int64_t shape[2], stride[2];
    m->type = type_of(t);
    if (want < 0 && (m->type < 0 || m->type > BF16)) {
        PyErr_Format(PyExc_TypeError, "%s must be a float32, float16 or bfloat16 tensor", name);
        return -1;
    }
    if (layout(t, 2, shape, stride) != 0) {
        PyErr_Format(PyExc_ValueError, "%s must be a 2-D tensor", name);
        return -1;
    }
    if (want >= 0 && m->type != want) return wrong_type(t, name, want);
    if (!on_gpu(t)) {
        PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", name);
        return -1;
    }
    m->rows = shape[0];
    m->cols = shape[1];
    m->ld = stride[0];
    if (stride[1] != 1 && m->cols > 1) {
        PyErr_Format(PyExc_ValueError, "%s must have unit column stride", name);
        return -1;
    }
    if (m->ld < m->cols) {
        if (m->rows > 1) {
            PyErr_Format(PyExc_ValueError, "%s has overlapping rows", name);
            return -1;
        }
        m->ld = m->cols; /* the pitch of a single row is never used */
    }
    if (same_device(t, name, device) != 0) return -1;
    return address(t, &m->ptr);
}

static int matrix_like(PyObject *t, const char *name, int want, const Mat *like, Mat *m, int64_t *device)
{
    if (matrix(t, name, want, m, device) != 0) return -1;
    if (m->rows != like->rows || m->cols != like->cols) {
        PyErr_Format(PyExc_ValueError, "shape mismatch: %s (%lld, %lld), expected (%lld, %lld)", name,
                     (long long)m->rows, (long long)m->cols, (long long)like->rows, (long long)like->cols);
        return -1;
    }
    return 0;
}

static int vector(PyObject *t, const char *name, int want, int64_t n, void **ptr, int64_t *device)
{
    int64_t shape, stride;
    if (layout(t, 1, &shape, &stride) != 0 || shape != n) {
        PyErr_Format(PyExc_ValueError, "%s must be a 1-D tensor of %lld", name, (long long)n);
        return -1;
    }
    if (type_of(t) != want) return wrong_type(t, name, want);
    if (!on_gpu(t) || (n > 1 && stride != 1)) {
        PyErr_Format(PyExc_ValueError, "%s must be a contiguous CUDA tensor", name);
        return -1;
    }
    if (same_device(t, name, device) != 0) return -1;
    return address(t, ptr);
}

/* ---- the stream, entry points and results */

/* None: the current device's current stream; a Stream; or a handle.  The
 * tensors have to be on the current device, which is where kernels are launched. */
static int stream_of(PyObject *s, int64_t device, void **out)
{
    PyObject *h, *dev = PyObject_CallNoArgs(g_get_device);
    if (!dev) return -1;
    const int64_t current = PyLong_AsLongLong(dev);
    if (current != device) {
        if (!PyErr_Occurred())
            PyErr_Format(PyExc_ValueError, "the tensors are on cuda:%lld, the current device is cuda:%lld",
                         (long long)device, (long long)current);
        Py_DECREF(dev);
        return -1;
    }
    if (s == Py_None) {
        h = PyObject_CallOneArg(g_raw_stream, dev);
    } else if (PyLong_Check(s)) {
        Py_INCREF(s);
        h = s;
    } else {
        h = PyObject_GetAttr(s, s_cuda_stream);
    }
    Py_DECREF(dev);
    if (!h) return -1;
    *out = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    return *out == NULL && PyErr_Occurred() ? -1 : 0;
}

static int arity(const char *name, Py_ssize_t got, Py_ssize_t want)
{
    if (got == want) return 0;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, got);
    return -1;
}

static int entry(PyObject *a, void **fn)
{
    *fn = PyLong_AsVoidPtr(a);
    if (*fn) return 0;
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null entry point");
    return -1;
}

/* Raises the binding's error for a status that is not OK. */
static int failed(int st, const char *name)
{
    if (st == 0) return 0;
    PyObject *e = PyObject_CallFunction(g_error, "is", st, name);
    if (e) {
        PyErr_SetObject((PyObject *)Py_TYPE(e), e);
        Py_DECREF(e);
    }
    return 1;
}

/* ---- the calls: (entry point, the call's arguments in order, stream) */

typedef int (*quantize_fn)(int64_t, int64_t, const void *, int64_t, int, int8_t *, int64_t, float *, void *);
typedef int (*rmsnorm_fn)(int64_t, int64_t, const void *, int64_t, const void *, int64_t, const void *, int, float, int,
                          void *, int64_t, int8_t *, int64_t, float *, void *);
typedef int (*swiglu_fn)(int64_t, int64_t, const void *, int64_t, const void *, int64_t, int, int8_t *, int64_t, float *,
                         void *);
typedef int (*dequantize_fn)(int64_t, int64_t, const int8_t *, int64_t, const float *, void *, int64_t, int, void *);
typedef int (*gemm_fn)(int64_t, int64_t, int64_t, const int8_t *, int64_t, const float *, const int8_t *, int64_t,
                       const float *, const float *, float, void *, int64_t, int, void *);

static PyObject *quantize_i8(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Mat x, q;
    void *fn, *scale, *stream;
    int64_t device = -1;
    int st;
    (void)self;
    if (arity("quantize_i8", n, 5) || entry(a[0], &fn) || matrix(a[1], "X", -1, &x, &device) ||
        matrix_like(a[2], "Q", I8, &x, &q, &device) || vector(a[3], "scale", F32, x.rows, &scale, &device) ||
        stream_of(a[4], device, &stream))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = ((quantize_fn)fn)(x.rows, x.cols, x.ptr, x.ld, x.type, q.ptr, q.ld, scale, stream);
    Py_END_ALLOW_THREADS
    return failed(st, "quantize_i8") ? NULL : PyTuple_Pack(2, a[2], a[3]);
}

static PyObject *rmsnorm_i8(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Mat x, q, r = {0}, h = {0};
    void *fn, *gamma, *scale, *stream;
    int64_t device = -1;
    int st;
    (void)self;
    if (arity("rmsnorm_i8", n, 9) || entry(a[0], &fn) || matrix(a[1], "X", -1, &x, &device) ||
        matrix_like(a[3], "Q", I8, &x, &q, &device) ||
        (a[5] != Py_None && matrix_like(a[5], "residual", x.type, &x, &r, &device)) ||
        (a[6] != Py_None && matrix_like(a[6], "H", x.type, &x, &h, &device)))
        return NULL;
    /* the weights: FP32, or the rows' type */
    const int gtype = type_of(a[2]) == F32 ? F32 : x.type;
    const double eps = PyFloat_AsDouble(a[7]);
    if ((eps == -1.0 && PyErr_Occurred()) || vector(a[2], "gamma", gtype, x.cols, &gamma, &device) ||
        vector(a[4], "scale", F32, x.rows, &scale, &device) || stream_of(a[8], device, &stream))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = ((rmsnorm_fn)fn)(x.rows, x.cols, x.ptr, x.ld, r.ptr, r.ld, gamma, gtype, (float)eps, x.type, h.ptr, h.ld, q.ptr,
                          q.ld, scale, stream);
    Py_END_ALLOW_THREADS
    return failed(st, "rmsnorm_i8") ? NULL : PyTuple_Pack(2, a[3], a[4]);
}

static PyObject *swiglu_i8(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Mat g, u, q;
    void *fn, *scale, *stream;
    int64_t device = -1;
    int st;
    (void)self;
    if (arity("swiglu_i8", n, 6) || entry(a[0], &fn) || matrix(a[1], "G", -1, &g, &device) ||
        matrix_like(a[2], "U", g.type, &g, &u, &device) || matrix_like(a[3], "Q", I8, &g, &q, &device) ||
        vector(a[4], "scale", F32, g.rows, &scale, &device) || stream_of(a[5], device, &stream))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = ((swiglu_fn)fn)(g.rows, g.cols, g.ptr, g.ld, u.ptr, u.ld, g.type, q.ptr, q.ld, scale, stream);
    Py_END_ALLOW_THREADS
    return failed(st, "swiglu_i8") ? NULL : PyTuple_Pack(2, a[3], a[4]);
}

static PyObject *dequantize_i8(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Mat x, q;
    void *fn, *scale, *stream;
    int64_t device = -1;
    int st;
    (void)self;
    if (arity("dequantize_i8", n, 5) || entry(a[0], &fn) || matrix(a[3], "X", -1, &x, &device) ||
        matrix_like(a[1], "Q", I8, &x, &q, &device) || vector(a[2], "scale", F32, x.rows, &scale, &device) ||
        stream_of(a[4], device, &stream))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = ((dequantize_fn)fn)(x.rows, x.cols, q.ptr, q.ld, scale, x.ptr, x.ld, x.type, stream);
    Py_END_ALLOW_THREADS
    if (failed(st, "dequantize_i8")) return NULL;
    Py_INCREF(a[3]);
    return a[3];
}

static PyObject *gemm_i8_tn(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Mat A, B, C;
    void *fn, *sa, *sb, *bias = NULL, *stream;
    int64_t device = -1;
    int st;
    (void)self;
    if (arity("gemm_i8_tn", n, 9) || entry(a[0], &fn) || matrix(a[3], "C", -1, &C, &device) ||
        matrix(a[1], "A", I8, &A, &device) || matrix(a[2], "B", I8, &B, &device))
        return NULL;
    if (A.rows != C.rows || B.rows != C.cols || A.cols != B.cols) {
        PyErr_Format(PyExc_ValueError, "shape mismatch: A (%lld, %lld), B (%lld, %lld), C (%lld, %lld)",
                     (long long)A.rows, (long long)A.cols, (long long)B.rows, (long long)B.cols, (long long)C.rows,
                     (long long)C.cols);
        return NULL;
    }
    const double beta = PyFloat_AsDouble(a[7]);
    if ((beta == -1.0 && PyErr_Occurred()) || vector(a[4], "scale_a", F32, C.rows, &sa, &device) ||
        vector(a[5], "scale_b", F32, C.cols, &sb, &device) ||
        (a[6] != Py_None && vector(a[6], "bias", F32, C.cols, &bias, &device)) || stream_of(a[8], device, &stream))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = ((gemm_fn)fn)(C.rows, C.cols, A.cols, A.ptr, A.ld, sa, B.ptr, B.ld, sb, bias, (float)beta, C.ptr, C.ld, C.type,
                       stream);
    Py_END_ALLOW_THREADS
    if (failed(st, "gemm_i8_tn")) return NULL;
    Py_INCREF(a[3]);
    return a[3];
}

/* ---- 8-bit floating point */

/* dgemm_f8 of include/dgemm.h */
typedef struct {
    void *data;
    int64_t ld;
    int type, block;
    float *scale;
    int64_t scale_row, scale_blk;
} F8;

/* What the three reads below end with: t on the GPU of the call, its address. */
static int placed(PyObject *t, const char *name, int64_t *device, void **ptr)
{
    if (!on_gpu(t)) {
        PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", name);
        return -1;
    }
    return same_device(t, name, device) != 0 ? -1 : address(t, ptr);
}

static int f8_type(PyObject *t, const char *name, int *type)
{
    const int code = type_of(t);
    *type = code - E4M3;
    if (code == E4M3 || code == E5M2) return 0;
    PyErr_Format(PyExc_TypeError, "%s must be a float8_e4m3fn or float8_e5m2 tensor", name);
    return -1;
}

/* The scales of `rows` x `cols` values, one for each 128 columns of a row or (where
 * rows <= 1 both are the same) of a band of 128; sets q's block and strides.  `written`:
 * each scale has a place of its own. */
static int f8_scale(PyObject *t, const char *name, int64_t rows, int64_t cols, int written, F8 *q, int64_t *device)
{
    int64_t shape[2], stride[2];
    const int64_t bands = (rows + 127) / 128, blocks = (cols + 127) / 128;
    if (type_of(t) != F32) return wrong_type(t, name, F32);
    if (layout(t, 2, shape, stride) != 0 || shape[1] != blocks || (shape[0] != rows && shape[0] != bands)) {
        PyErr_Format(PyExc_ValueError, "%s must be a 2-D tensor of (%lld or %lld, %lld)", name, (long long)rows,
                     (long long)bands, (long long)blocks);
        return -1;
    }
    q->block = shape[0] == rows ? 1 : 128;
    q->scale_row = shape[0] > 1 ? stride[0] : 1;
    q->scale_blk = shape[1] > 1 ? stride[1] : 1;
    if (written && shape[0] > 1 && shape[1] > 1) {
        const int64_t a = q->scale_row, b = q->scale_blk;
        if (a < 1 || b < 1 || !(a >= b * shape[1] || b >= a * shape[0])) {
            PyErr_Format(PyExc_ValueError, "%s has overlapping elements", name);
            return -1;
        }
    }
    return placed(t, name, device, (void **)&q->scale);
}

/* A matrix in 8-bit floating point and its scales; rows, cols < 0: of any size. */
static int f8_matrix(PyObject *t, const char *name, PyObject *scale, const char *scale_name, int64_t rows, int64_t cols,
                     int written, F8 *q, int64_t *got_rows, int64_t *got_cols, int64_t *device)
{
    Mat m;
    if (f8_type(t, name, &q->type) != 0 || matrix(t, name, E4M3 + q->type, &m, device) != 0) return -1;
    if ((rows >= 0 && m.rows != rows) || (cols >= 0 && m.cols != cols)) {
        PyErr_Format(PyExc_ValueError, "shape mismatch: %s (%lld, %lld), expected (%lld, %lld)", name, (long long)m.rows,
                     (long long)m.cols, (long long)(rows >= 0 ? rows : m.rows), (long long)(cols >= 0 ? cols : m.cols));
        return -1;
    }
    q->data = m.ptr;
    q->ld = m.ld;
    if (got_rows) *got_rows = m.rows;
    if (got_cols) *got_cols = m.cols;
    return f8_scale(scale, scale_name, m.rows, m.cols, written, q, device);
}

/* A contiguous tensor of `want` and of n0 (x n1, if n1 >= 0) elements. */
static int integers(PyObject *t, const char *name, int want, int64_t n0, int64_t n1, void **ptr, int64_t *device)
{
    int64_t shape[2], stride[2];
    const Py_ssize_t dims = n1 < 0 ? 1 : 2;
    if (layout(t, dims, shape, stride) != 0 || shape[0] != n0 || (dims == 2 && shape[1] != n1)) {
        if (dims == 1)
            PyErr_Format(PyExc_ValueError, "%s must be a 1-D tensor of %lld", name, (long long)n0);
        else
            PyErr_Format(PyExc_ValueError, "%s must be a 2-D tensor of (%lld, %lld)", name, (long long)n0, (long long)n1);
        return -1;
    }
    if (type_of(t) != want) return wrong_type(t, name, want);
    const int inner = dims == 1 ? 0 : 1;
    if ((shape[inner] > 1 && stride[inner] != 1) || (dims == 2 && shape[0] > 1 && shape[1] > 0 && stride[0] != shape[1])) {
        PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
        return -1;
    }
    return placed(t, name, device, ptr);
}

typedef int (*quantize_f8_fn)(int64_t, int64_t, const void *, int64_t, int, int, const F8 *, void *);
typedef int (*swiglu_f8_fn)(int64_t, int64_t, const void *, int64_t, const void *, int64_t, int, const F8 *, void *);
typedef int (*dequantize_f8_fn)(int64_t, int64_t, const F8 *, void *, int64_t, int, void *);
typedef int (*gemm_f8_fn)(int64_t, int64_t, int64_t, const F8 *, const F8 *, const float *, float, void *, int64_t, int, void *);
typedef int (*experts_f8_fn)(int64_t, int64_t, int64_t, int, const int32_t *, const F8 *, const F8 *, int64_t, int64_t, void *,
                             int64_t, int, void *);
typedef int (*sort_fn)(int64_t, int64_t, int, const void *, int, int32_t *, int32_t *, void *);
typedef int (*gather_fn)(int64_t, int64_t, int64_t, const void *, int64_t, int, const int32_t *, int64_t, void *, int64_t, void *);
typedef int (*gather_f8_fn)(int64_t, int64_t, int64_t, const void *, int64_t, int, const int32_t *, int64_t, const F8 *, void *);
typedef int (*combine_fn)(int64_t, int64_t, int64_t, const void *, int64_t, int64_t, int, const int32_t *, const float *, float,
                          void *, int64_t, void *);
typedef int (*combine_grad_fn)(int64_t, int64_t, int64_t, const void *, int64_t, const void *, int64_t, int64_t, int,
                               const int32_t *, const float *, void *, int64_t, float *, void *);

static PyObject *quantize_f8(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Mat x;
    F8 q;
    void *fn, *stream;
    int64_t device = -1;
    int st;
    (void)self;
    if (arity("quantize_f8", n, 6) || entry(a[0], &fn) || matrix(a[1], "X", -1, &x, &device)) return NULL;
    const int transposed = PyObject_IsTrue(a[4]);
    if (transposed < 0 || f8_matrix(a[2], "Q", a[3], "scale", transposed ? x.cols : x.rows, transposed ? x.rows : x.cols, 1, &q,
                                    NULL, NULL, &device) ||
        stream_of(a[5], device, &stream))
        return NULL;
    if (transposed && q.block != 1) {
        PyErr_SetString(PyExc_ValueError, "a transposed quantisation has a scale for each row of Q");
        return NULL;
    }
    Py_BEGIN_ALLOW_THREADS
    st = ((quantize_f8_fn)fn)(x.rows, x.cols, x.ptr, x.ld, x.type, transposed, &q, stream);
    Py_END_ALLOW_THREADS
    return failed(st, "quantize_f8") ? NULL : PyTuple_Pack(2, a[2], a[3]);
}

/* Whether an operand has a scale a row, where the call knows no other. */
static int a_scale_a_row(const F8 *q, const char *name)
{
    if (q->block == 1) return 0;
    PyErr_Format(PyExc_ValueError, "%s must have a row for each row it scales", name);
    return -1;
}

static PyObject *swiglu_f8(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Mat g, u;
    F8 q;
    void *fn, *stream;
    int64_t device = -1;
    int st;
    (void)self;
    if (arity("swiglu_f8", n, 6) || entry(a[0], &fn) || matrix(a[1], "G", -1, &g, &device) ||
        matrix_like(a[2], "U", g.type, &g, &u, &device) ||
        f8_matrix(a[3], "Q", a[4], "scale", g.rows, g.cols, 1, &q, NULL, NULL, &device) || a_scale_a_row(&q, "scale") ||
        stream_of(a[5], device, &stream))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = ((swiglu_f8_fn)fn)(g.rows, g.cols, g.ptr, g.ld, u.ptr, u.ld, g.type, &q, stream);
    Py_END_ALLOW_THREADS
    return failed(st, "swiglu_f8") ? NULL : PyTuple_Pack(2, a[3], a[4]);
}

static PyObject *dequantize_f8(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Mat x;
    F8 q;
    void *fn, *stream;
    int64_t device = -1;
    int st;
    (void)self;
    if (arity("dequantize_f8", n, 5) || entry(a[0], &fn) || matrix(a[3], "X", -1, &x, &device) ||
        f8_matrix(a[1], "Q", a[2], "scale", x.rows, x.cols, 0, &q, NULL, NULL, &device) || stream_of(a[4], device, &stream))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = ((dequantize_f8_fn)fn)(x.rows, x.cols, &q, x.ptr, x.ld, x.type, stream);
    Py_END_ALLOW_THREADS
    if (failed(st, "dequantize_f8")) return NULL;
    Py_INCREF(a[3]);
    return a[3];
}

static PyObject *gemm_f8_tn(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Mat C;
    F8 A, B;
    void *fn, *bias = NULL, *stream;
    int64_t device = -1, K;
    int st;
    (void)self;
    if (arity("gemm_f8_tn", n, 9) || entry(a[0], &fn) || matrix(a[3], "C", -1, &C, &device) ||
        f8_matrix(a[1], "A", a[4], "scale_a", C.rows, -1, 0, &A, NULL, &K, &device) ||
        f8_matrix(a[2], "B", a[5], "scale_b", C.cols, K, 0, &B, NULL, NULL, &device))
        return NULL;
    const double beta = PyFloat_AsDouble(a[7]);
    if ((beta == -1.0 && PyErr_Occurred()) || (a[6] != Py_None && vector(a[6], "bias", F32, C.cols, &bias, &device)) ||
        stream_of(a[8], device, &stream))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = ((gemm_f8_fn)fn)(C.rows, C.cols, K, &A, &B, bias, (float)beta, C.ptr, C.ld, C.type, stream);
    Py_END_ALLOW_THREADS
    if (failed(st, "gemm_f8_tn")) return NULL;
    Py_INCREF(a[3]);
    return a[3];
}

static PyObject *gemm_f8_tn_experts(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Mat C;
    F8 A, B;
    void *fn, *offsets, *stream;
    int64_t device = -1, K, shape[3], stride[3];
    int st;
    (void)self;
    if (arity("gemm_f8_tn_experts", n, 8) || entry(a[0], &fn) || matrix(a[3], "C", -1, &C, &device) ||
        f8_matrix(a[1], "A", a[4], "scale_a", C.rows, -1, 0, &A, NULL, &K, &device) || a_scale_a_row(&A, "scale_a") ||
        f8_type(a[2], "B", &B.type))
        return NULL;
    if (layout(a[2], 3, shape, stride) != 0 || shape[0] < 1 || shape[1] != C.cols || shape[2] != K) {
        PyErr_Format(PyExc_ValueError, "B must be a 3-D tensor of (experts, %lld, %lld)", (long long)C.cols, (long long)K);
        return NULL;
    }
    if (shape[2] > 1 && stride[2] != 1) {
        PyErr_SetString(PyExc_ValueError, "B must have unit column stride");
        return NULL;
    }
    const int64_t experts = shape[0], b_stride = experts > 1 ? stride[0] : 0;
    B.ld = shape[1] > 1 ? stride[1] : shape[2];
    if (B.ld < K || b_stride < 0) {
        PyErr_SetString(PyExc_ValueError, "B has overlapping rows");
        return NULL;
    }
    const int64_t bands = (C.cols + 127) / 128, blocks = (K + 127) / 128;
    if (type_of(a[5]) != F32) {
        wrong_type(a[5], "scale_b", F32);
        return NULL;
    }
    if (layout(a[5], 3, shape, stride) != 0 || shape[0] != experts || shape[2] != blocks ||
        (shape[1] != C.cols && shape[1] != bands)) {
        PyErr_Format(PyExc_ValueError, "scale_b must be a 3-D tensor of (%lld, %lld or %lld, %lld)", (long long)experts,
                     (long long)C.cols, (long long)bands, (long long)blocks);
        return NULL;
    }
    B.block = shape[1] == C.cols ? 1 : 128;
    B.scale_row = shape[1] > 1 ? stride[1] : 1;
    B.scale_blk = shape[2] > 1 ? stride[2] : 1;
    const int64_t scale_stride = experts > 1 ? stride[0] : 0;
    if (placed(a[2], "B", &device, &B.data) || placed(a[5], "scale_b", &device, (void **)&B.scale) ||
        integers(a[6], "offsets", I32, experts + 1, -1, &offsets, &device) || stream_of(a[7], device, &stream))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = ((experts_f8_fn)fn)(C.rows, C.cols, K, experts > INT32_MAX ? 0 : (int)experts, offsets, &A, &B, b_stride, scale_stride, C.ptr, C.ld, C.type,
                             stream);
    Py_END_ALLOW_THREADS
    if (failed(st, "gemm_f8_tn_experts")) return NULL;
    Py_INCREF(a[3]);
    return a[3];
}

/* ---- tokens by expert */

/* A matrix of pairs (token, choice), contiguous; its type. */
static int pairs(PyObject *t, const char *name, int64_t *tokens, int64_t *top, void **ptr, int *type, int64_t *device)
{
    int64_t shape[2], stride[2];
    if (layout(t, 2, shape, stride) != 0) {
        PyErr_Format(PyExc_ValueError, "%s must be a 2-D tensor", name);
        return -1;
    }
    *type = type_of(t);
    if (*type != I32 && *type != I64) {
        PyErr_Format(PyExc_TypeError, "%s must be an int32 or int64 tensor", name);
        return -1;
    }
    *tokens = shape[0];
    *top = shape[1];
    return integers(t, name, *type, shape[0], shape[1], ptr, device);
}

static int positions(PyObject *t, int64_t tokens, int64_t *top, void **ptr, int64_t *device)
{
    int64_t got;
    int type;
    if (pairs(t, "position", &got, top, ptr, &type, device) != 0) return -1;
    if (type != I32) return wrong_type(t, "position", I32);
    if (got == tokens) return 0;
    PyErr_Format(PyExc_ValueError, "position is for %lld tokens, expected %lld", (long long)got, (long long)tokens);
    return -1;
}

static PyObject *sort_by_expert(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    void *fn, *ids, *offsets, *position, *stream;
    int64_t device = -1, tokens, top, entries, step;
    int type, st;
    (void)self;
    if (arity("sort_by_expert", n, 5) || entry(a[0], &fn) || pairs(a[1], "experts", &tokens, &top, &ids, &type, &device))
        return NULL;
    if (layout(a[2], 1, &entries, &step) != 0 || entries < 2) {
        PyErr_SetString(PyExc_ValueError, "offsets must be a 1-D tensor of the number of experts + 1");
        return NULL;
    }
    if (integers(a[2], "offsets", I32, entries, -1, &offsets, &device) ||
        integers(a[3], "position", I32, tokens, top, &position, &device) || stream_of(a[4], device, &stream))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = ((sort_fn)fn)(tokens, top, entries - 1 > INT32_MAX ? 0 : (int)(entries - 1), ids, type == I64 ? 8 : 4, offsets,
                       position, stream);
    Py_END_ALLOW_THREADS
    return failed(st, "sort_by_expert") ? NULL : PyTuple_Pack(2, a[2], a[3]);
}

static PyObject *gather_by_expert(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Mat x, y;
    void *fn, *position, *stream;
    int64_t device = -1, top;
    int st;
    (void)self;
    if (arity("gather_by_expert", n, 5) || entry(a[0], &fn) || matrix(a[1], "X", -1, &x, &device) ||
        positions(a[2], x.rows, &top, &position, &device) || matrix(a[3], "Y", x.type, &y, &device))
        return NULL;
    if (y.cols != x.cols) {
        PyErr_Format(PyExc_ValueError, "shape mismatch: Y has %lld columns, X %lld", (long long)y.cols, (long long)x.cols);
        return NULL;
    }
    if (stream_of(a[4], device, &stream)) return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = ((gather_fn)fn)(x.rows, top, x.cols, x.ptr, x.ld, x.type, position, y.rows, y.ptr, y.ld, stream);
    Py_END_ALLOW_THREADS
    if (failed(st, "gather_by_expert")) return NULL;
    Py_INCREF(a[3]);
    return a[3];
}

static PyObject *gather_by_expert_f8(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Mat x;
    F8 q;
    void *fn, *position, *stream;
    int64_t device = -1, top, rows;
    int st;
    (void)self;
    if (arity("gather_by_expert_f8", n, 6) || entry(a[0], &fn) || matrix(a[1], "X", -1, &x, &device) ||
        positions(a[2], x.rows, &top, &position, &device) ||
        f8_matrix(a[3], "Q", a[4], "scale", -1, x.cols, 1, &q, &rows, NULL, &device) || a_scale_a_row(&q, "scale") ||
        stream_of(a[5], device, &stream))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = ((gather_f8_fn)fn)(x.rows, top, x.cols, x.ptr, x.ld, x.type, position, rows, &q, stream);
    Py_END_ALLOW_THREADS
    return failed(st, "gather_by_expert_f8") ? NULL : PyTuple_Pack(2, a[3], a[4]);
}

static PyObject *combine_experts(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Mat x, y;
    void *fn, *position, *weights = NULL, *stream;
    int64_t device = -1, top;
    int st;
    (void)self;
    if (arity("combine_experts", n, 7) || entry(a[0], &fn) || matrix(a[4], "X", -1, &x, &device) ||
        matrix(a[1], "Y", x.type, &y, &device) || positions(a[2], x.rows, &top, &position, &device) ||
        (a[3] != Py_None && integers(a[3], "weights", F32, x.rows, top, &weights, &device)))
        return NULL;
    if (y.cols != x.cols) {
        PyErr_Format(PyExc_ValueError, "shape mismatch: Y has %lld columns, X %lld", (long long)y.cols, (long long)x.cols);
        return NULL;
    }
    const double beta = PyFloat_AsDouble(a[5]);
    if ((beta == -1.0 && PyErr_Occurred()) || stream_of(a[6], device, &stream)) return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = ((combine_fn)fn)(x.rows, top, x.cols, y.ptr, y.ld, y.rows, x.type, position, weights, (float)beta, x.ptr, x.ld, stream);
    Py_END_ALLOW_THREADS
    if (failed(st, "combine_experts")) return NULL;
    Py_INCREF(a[4]);
    return a[4];
}

static PyObject *combine_experts_grad(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Mat dx, y, dy;
    void *fn, *position, *weights, *dw, *stream;
    int64_t device = -1, top;
    int st;
    (void)self;
    if (arity("combine_experts_grad", n, 8) || entry(a[0], &fn) || matrix(a[1], "dX", -1, &dx, &device) ||
        matrix(a[2], "Y", dx.type, &y, &device) || positions(a[3], dx.rows, &top, &position, &device) ||
        integers(a[4], "weights", F32, dx.rows, top, &weights, &device) || matrix_like(a[5], "dY", dx.type, &y, &dy, &device) ||
        integers(a[6], "dweights", F32, dx.rows, top, &dw, &device))
        return NULL;
    if (y.cols != dx.cols) {
        PyErr_Format(PyExc_ValueError, "shape mismatch: Y has %lld columns, dX %lld", (long long)y.cols, (long long)dx.cols);
        return NULL;
    }
    if (stream_of(a[7], device, &stream)) return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = ((combine_grad_fn)fn)(dx.rows, top, dx.cols, dx.ptr, dx.ld, y.ptr, y.ld, y.rows, dx.type, position, weights, dy.ptr,
                               dy.ld, dw, stream);
    Py_END_ALLOW_THREADS
    return failed(st, "combine_experts_grad") ? NULL : PyTuple_Pack(2, a[5], a[6]);
}

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, "setup(float32, float16, bfloat16, int8, get_device, raw_stream, error[, float8_e4m3fn, float8_e5m2, int32, int64])"},
    {"quantize_i8", (PyCFunction)(void (*)(void))quantize_i8, METH_FASTCALL, "(entry, X, Q, scale, stream)"},
    {"rmsnorm_i8", (PyCFunction)(void (*)(void))rmsnorm_i8, METH_FASTCALL,
     "(entry, X, gamma, Q, scale, residual, H, eps, stream)"},
    {"swiglu_i8", (PyCFunction)(void (*)(void))swiglu_i8, METH_FASTCALL, "(entry, G, U, Q, scale, stream)"},
    {"dequantize_i8", (PyCFunction)(void (*)(void))dequantize_i8, METH_FASTCALL, "(entry, Q, scale, X, stream)"},
    {"gemm_i8_tn", (PyCFunction)(void (*)(void))gemm_i8_tn, METH_FASTCALL,
     "(entry, A, B, C, scale_a, scale_b, bias, beta, stream)"},
    {"quantize_f8", (PyCFunction)(void (*)(void))quantize_f8, METH_FASTCALL,
     "(entry, X, Q, scale, transposed, stream)"},
    {"swiglu_f8", (PyCFunction)(void (*)(void))swiglu_f8, METH_FASTCALL,
     "(entry, G, U, Q, scale, stream)"},
    {"dequantize_f8", (PyCFunction)(void (*)(void))dequantize_f8, METH_FASTCALL,
     "(entry, Q, scale, X, stream)"},
    {"gemm_f8_tn", (PyCFunction)(void (*)(void))gemm_f8_tn, METH_FASTCALL,
     "(entry, A, B, C, scale_a, scale_b, bias, beta, stream)"},
    {"gemm_f8_tn_experts", (PyCFunction)(void (*)(void))gemm_f8_tn_experts, METH_FASTCALL,
     "(entry, A, B, C, scale_a, scale_b, offsets, stream)"},
    {"sort_by_expert", (PyCFunction)(void (*)(void))sort_by_expert, METH_FASTCALL,
     "(entry, experts, offsets, position, stream)"},
    {"gather_by_expert", (PyCFunction)(void (*)(void))gather_by_expert, METH_FASTCALL,
     "(entry, X, position, Y, stream)"},
    {"gather_by_expert_f8", (PyCFunction)(void (*)(void))gather_by_expert_f8, METH_FASTCALL,
     "(entry, X, position, Q, scale, stream)"},
    {"combine_experts", (PyCFunction)(void (*)(void))combine_experts, METH_FASTCALL,
     "(entry, Y, position, weights, X, beta, stream)"},
    {"combine_experts_grad", (PyCFunction)(void (*)(void))combine_experts_grad, METH_FASTCALL,
     "(entry, dX, Y, position, weights, dY, dweights, stream)"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_i8_calls", "Marshalling of the 8-bit calls.", -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__i8_calls(void)
{
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_is_cuda = PyUnicode_InternFromString("is_cuda");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    if (!s_shape || !s_stride || !s_dtype || !s_is_cuda || !s_get_device || !s_data_ptr || !s_cuda_stream) return NULL;
    return PyModule_Create(&module);
}
