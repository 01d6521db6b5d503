/* The layer operators' calls from Python, without ctypes in between: converting
 * their 12 to 18 arguments there costs 1.4 us and finding the tensors' addresses
 * another 1.2, as much as the launch itself.  Each function here takes the
 * arguments of its C entry point in order (include/ar.h) and returns the status
 * code.  A pointer may be None (NULL), an address, or an object with data_ptr();
 * a stream None (the caller's current stream), a cudaStream_t as an integer, or
 * an object with cuda_stream. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "ar.h"

static PyObject *name_data_ptr, *name_cuda_stream;
static PyObject *raw_stream, *current_device;      /* torch's, once it has CUDA up */

/* One call's arguments, taken in order; `bad` once one did not convert. */
typedef struct {
    PyObject *const *arg;
    Py_ssize_t left;
    int bad;
} Args;

static PyObject *take(Args *a) {
    --a->left;
    return *a->arg++;
}

static void *pointer(Args *a) {
    PyObject *o = take(a), *address;
    void *p;
    if (a->bad || o == Py_None)
        return NULL;
    if (PyLong_Check(o)) {
        p = PyLong_AsVoidPtr(o);
    } else {
        address = PyObject_CallMethodNoArgs(o, name_data_ptr);
        if (!address) {
            a->bad = 1;
            return NULL;
        }
        p = PyLong_AsVoidPtr(address);
        Py_DECREF(address);
    }
    if (!p && PyErr_Occurred())
        a->bad = 1;
    return p;
}

static size_t size(Args *a) {
    PyObject *o = take(a);
    size_t n = 0;
    if (!a->bad) {
        n = PyLong_AsSize_t(o);
        a->bad = n == (size_t)-1 && PyErr_Occurred();
    }
    return n;
}

static int integer(Args *a) {
    PyObject *o = take(a);
    long n = 0;
    if (!a->bad) {
        n = PyLong_AsLong(o);
        a->bad = n == -1 && PyErr_Occurred();
        if (!a->bad && n != (int)n) {
            PyErr_SetString(PyExc_OverflowError, "argument does not fit a C int");
            a->bad = 1;
        }
    }
    return (int)n;
}

static float real(Args *a) {
    PyObject *o = take(a);
    double v = 0.0;
    if (!a->bad) {
        v = PyFloat_AsDouble(o);
        a->bad = v == -1.0 && PyErr_Occurred();
    }
    return (float)v;
}

/* torch's current stream: its raw lookup takes a tenth of the time of building a
 * Stream object; where torch has none, the public way. */
static PyObject *torch_stream(void) {
    PyObject *torch = NULL, *cuda = NULL, *up = NULL, *core = NULL, *s = NULL, *r = NULL, *device;
    if (!raw_stream) {
        torch = PyImport_ImportModule("torch");
        cuda = torch ? PyObject_GetAttrString(torch, "cuda") : NULL;
        up = cuda ? PyObject_CallMethod(cuda, "is_initialized", NULL) : NULL;
        core = up ? PyObject_GetAttrString(torch, "_C") : NULL;
        if (core && up == Py_True) {
            raw_stream = PyObject_GetAttrString(core, "_cuda_getCurrentRawStream");
            current_device = PyObject_GetAttrString(core, "_cuda_getDevice");
            if (!raw_stream || !current_device) {
                PyErr_Clear();
                Py_CLEAR(raw_stream);
                Py_CLEAR(current_device);
            }
        }
        if (core && !raw_stream) {
            s = PyObject_CallMethod(cuda, "current_stream", NULL);
            r = s ? PyObject_GetAttr(s, name_cuda_stream) : NULL;
        }
        Py_XDECREF(s);
        Py_XDECREF(core);
        Py_XDECREF(up);
        Py_XDECREF(cuda);
        Py_XDECREF(torch);
        if (!raw_stream)
            return r;
    }
    device = PyObject_CallNoArgs(current_device);
    if (!device)
        return NULL;
    r = PyObject_CallOneArg(raw_stream, device);
    Py_DECREF(device);
    return r;
}

static cudaStream_t stream(Args *a) {
    PyObject *o = take(a), *n;
    void *p;
    if (a->bad)
        return NULL;
    if (PyLong_Check(o)) {
        n = Py_NewRef(o);
    } else {
        n = o == Py_None ? torch_stream() : PyObject_GetAttr(o, name_cuda_stream);
        if (!n) {
            a->bad = 1;
            return NULL;
        }
    }
    p = PyLong_AsVoidPtr(n);
    Py_DECREF(n);
    a->bad = !p && PyErr_Occurred();
    return (cudaStream_t)p;
}

/* Opens a call of n arguments; the arguments are evaluated one after the other
 * into locals, because C leaves the order within a call open. */
#define BEGIN(n)                                                                        \
    Args a = {args, nargs, 0};                                                          \
    (void)self;                                                                         \
    if (nargs != (n)) {                                                                 \
        PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", (n), nargs);  \
        return NULL;                                                                    \
    }
#define P(name) void *name = pointer(&a)
#define Z(name) const size_t name = size(&a)
#define I(name) const int name = integer(&a)
/* Other threads run during the call, as they do with ctypes: a launch blocks while
 * the queue is full, and the queue may wait for a host callback into Python.
 * (One row of ar_rmsnorm: 3.77 to 3.93 us a call so, 3.62 to 3.73 with the lock
 * kept; decode order and dispatch 5.7 either way.) */
#define CALL(f)                                                                         \
    int status;                                                                         \
    if (a.bad)                                                                          \
        return NULL;                                                                    \
    Py_BEGIN_ALLOW_THREADS                                                              \
    status = f;                                                                         \
    Py_END_ALLOW_THREADS                                                                \
    return PyLong_FromLong(status)

static PyObject *rmsnorm(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
    BEGIN(17)
    P(x); Z(ldx); P(res); Z(ldres); P(gamma);
    const float eps = real(&a);
    P(sum); Z(ldsum); P(y); Z(ldy); P(scale); P(rstd); Z(T); Z(H); I(dtype); I(out_dtype);
    const cudaStream_t s = stream(&a);
    CALL(ar_rmsnorm(x, ldx, res, ldres, gamma, eps, sum, ldsum, y, ldy, scale, rstd, T, H, dtype,
                    out_dtype, s));
}

static PyObject *rmsnorm_grad(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
    BEGIN(17)
    P(dy); Z(lddy); P(dsum); Z(lddsum); P(sum); Z(lds); P(gamma); P(rstd); P(dx); Z(lddx);
    P(dgamma); P(work); Z(work_bytes); Z(T); Z(H); I(dtype);
    const cudaStream_t s = stream(&a);
    CALL(ar_rmsnorm_grad(dy, lddy, dsum, lddsum, sum, lds, gamma, rstd, dx, lddx, dgamma, work,
                         work_bytes, T, H, dtype, s));
}

static PyObject *moe_route(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
    BEGIN(9)
    P(ids); I(ids_bytes); Z(T); I(K); I(E); P(offsets); P(row_of); P(src);
    const cudaStream_t s = stream(&a);
    CALL(ar_moe_route(ids, ids_bytes, T, K, E, offsets, row_of, src, s));
}

static PyObject *moe_dispatch(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
    BEGIN(13)
    P(x); Z(ldx); P(xscale); P(row_of); P(rows); Z(ldrows); P(rscale); Z(nrows); Z(T); I(K); Z(H);
    I(dtype);
    const cudaStream_t s = stream(&a);
    CALL(ar_moe_dispatch(x, ldx, xscale, row_of, rows, ldrows, rscale, nrows, T, K, H, dtype, s));
}

static PyObject *moe_return(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
    BEGIN(12)
    P(rows); Z(ldrows); Z(nrows); P(row_of); P(w); P(out); Z(ldout); Z(T); I(K); Z(H); I(dtype);
    const cudaStream_t s = stream(&a);
    CALL(ar_moe_return(rows, ldrows, nrows, row_of, w, out, ldout, T, K, H, dtype, s));
}

static PyObject *moe_return_grad(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
    BEGIN(15)
    P(dout); Z(lddout); P(rows); Z(ldrows); Z(nrows); P(row_of); P(w); P(drows); Z(lddrows); P(dw);
    Z(T); I(K); Z(H); I(dtype);
    const cudaStream_t s = stream(&a);
    CALL(ar_moe_return_grad(dout, lddout, rows, ldrows, nrows, row_of, w, drows, lddrows, dw, T, K,
                            H, dtype, s));
}

static PyObject *matmul8(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
    BEGIN(16)
    P(x); Z(lda); P(sa); P(b); Z(ldb); P(sb); P(offsets); I(E); P(d); Z(ldd); Z(M); Z(N); Z(K);
    I(out_dtype); P(word);
    const cudaStream_t s = stream(&a);
    CALL(ar_matmul8(x, lda, sa, b, ldb, sb, offsets, E, d, ldd, M, N, K, out_dtype, word, s));
}

#define FAST(name, f) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {
    FAST("ar_rmsnorm", rmsnorm),
    FAST("ar_rmsnorm_grad", rmsnorm_grad),
    FAST("ar_moe_route", moe_route),
    FAST("ar_moe_dispatch", moe_dispatch),
    FAST("ar_moe_return", moe_return),
    FAST("ar_moe_return_grad", moe_return_grad),
    FAST("ar_matmul8", matmul8),
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {
    PyModuleDef_HEAD_INIT, "_native", "The layer operators' calls (internal).", -1, methods,
    NULL, NULL, NULL, NULL,
};

PyMODINIT_FUNC PyInit__native(void) {
    name_data_ptr = PyUnicode_InternFromString("data_ptr");
    name_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    return name_data_ptr && name_cuda_stream ? PyModule_Create(&module) : NULL;
}
