/*
 * i8_calls.c -- CPython module _i8_calls: argument marshalling of the 8-bit
 * calls, in C.
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

enum { F32 = 0, F16 = 1, BF16 = 2, I8 = 3, kTypes = 4 }; /* 0..2: dgemm_type */
static PyObject *g_dtype[kTypes];
static PyObject *g_get_device, *g_raw_stream, *g_error;
static PyObject *s_shape, *s_stride, *s_dtype, *s_is_cuda, *s_get_device, *s_data_ptr, *s_cuda_stream;

static PyObject *setup(PyObject *self, PyObject *args)
{
    PyObject *d[kTypes], *dev, *raw, *err;
    (void)self;
    if (!PyArg_ParseTuple(args, "OOOOOOO", &d[0], &d[1], &d[2], &d[3], &dev, &raw, &err)) return NULL;
    for (int i = 0; i < kTypes; ++i) {
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
    if (want < 0 && (m->type < 0 || m->type == I8)) {
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

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, "setup(float32, float16, bfloat16, int8, get_device, raw_stream, error)"},
    {"quantize_i8", (PyCFunction)(void (*)(void))quantize_i8, METH_FASTCALL, "(entry, X, Q, scale, stream)"},
    {"rmsnorm_i8", (PyCFunction)(void (*)(void))rmsnorm_i8, METH_FASTCALL,
     "(entry, X, gamma, Q, scale, residual, H, eps, stream)"},
    {"swiglu_i8", (PyCFunction)(void (*)(void))swiglu_i8, METH_FASTCALL, "(entry, G, U, Q, scale, stream)"},
    {"dequantize_i8", (PyCFunction)(void (*)(void))dequantize_i8, METH_FASTCALL, "(entry, Q, scale, X, stream)"},
    {"gemm_i8_tn", (PyCFunction)(void (*)(void))gemm_i8_tn, METH_FASTCALL,
     "(entry, A, B, C, scale_a, scale_b, bias, beta, stream)"},
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
