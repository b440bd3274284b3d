/*
 * Argument marshalling for the entry points that a training step calls many
 * times, on small tensors too.  A call whose library side returns at once takes
 * 1.8 us through ctypes, with its dozen arguments, and 0.5 us through this
 * module (measured on an x86 host, wrapper included); a kernel's launch takes
 * 2.2 us.  It knows nothing but the signatures in zero.h; the functions'
 * addresses come from the binding, which has loaded the library.
 *
 * Each function takes its arguments by position and returns the library's code.
 * A pointer is an int, None (NULL) or an object with data_ptr() (a tensor).
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "zero.h"

static struct {
    __typeof__(&zero_embed) embed;
    __typeof__(&zero_embed_grad) embed_grad;
    __typeof__(&zero_dropout) dropout;
    __typeof__(&zero_mx4_quantize) quantize;
    __typeof__(&zero_mx4_dequantize) dequantize;
    __typeof__(&zero_mx4_matmul) matmul;
} lib;

static PyObject *data_ptr_name;

/* The arguments of one call; `bad` is set, with an exception, by the first
 * that is not what it should be. */
typedef struct {
    PyObject *const *at;
    int bad;
} args_t;

static void *pointer(args_t *a, int i)
{
    PyObject *o = a->at[i];
    void *p = NULL;
    if (a->bad || o == Py_None) return NULL;
    if (PyLong_Check(o)) {
        p = (void *)(uintptr_t)PyLong_AsUnsignedLongLong(o);
    } else {
        PyObject *v = PyObject_CallMethodNoArgs(o, data_ptr_name);
        if (v) {
            p = (void *)(uintptr_t)PyLong_AsUnsignedLongLong(v);
            Py_DECREF(v);
        }
    }
    if (PyErr_Occurred()) a->bad = 1;
    return p;
}

static int64_t whole(args_t *a, int i)
{
    long long v;
    if (a->bad) return 0;
    v = PyLong_AsLongLong(a->at[i]);
    if (v == -1 && PyErr_Occurred()) a->bad = 1;
    return v;
}

static int32_t small(args_t *a, int i)
{
    const int64_t v = whole(a, i);
    if (!a->bad && (v < INT32_MIN || v > INT32_MAX)) {
        PyErr_SetString(PyExc_OverflowError, "argument does not fit 32 bits");
        a->bad = 1;
    }
    return (int32_t)v;
}

static uint64_t word(args_t *a, int i)       /* modulo 2^64 */
{
    unsigned long long v;
    if (a->bad) return 0;
    v = PyLong_AsUnsignedLongLongMask(a->at[i]);
    if (v == (unsigned long long)-1 && PyErr_Occurred()) a->bad = 1;
    return v;
}

static int32_t truth(args_t *a, int i)
{
    int v;
    if (a->bad) return 0;
    v = PyObject_IsTrue(a->at[i]);
    if (v < 0) a->bad = 1;
    return v > 0;
}

static double real(args_t *a, int i)
{
    double v;
    if (a->bad) return 0.0;
    v = PyFloat_AsDouble(a->at[i]);
    if (v == -1.0 && PyErr_Occurred()) a->bad = 1;
    return v;
}

static int begin(args_t *a, PyObject *const *at, Py_ssize_t n, Py_ssize_t want, void *fn)
{
    a->at = at;
    a->bad = 0;
    if (!fn) {
        PyErr_SetString(PyExc_RuntimeError, "bind() comes first");
        return 0;
    }
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n);
        return 0;
    }
    return 1;
}

#define CALL(expression)            \
    do {                            \
        int rc;                     \
        if (a.bad) return NULL;     \
        Py_BEGIN_ALLOW_THREADS      \
        rc = (expression);          \
        Py_END_ALLOW_THREADS        \
        return PyLong_FromLong(rc); \
    } while (0)

static PyObject *embed(PyObject *self, PyObject *const *at, Py_ssize_t n)
{
    args_t a;
    if (!begin(&a, at, n, 14, (void *)lib.embed)) return NULL;
    const void *table = pointer(&a, 0);
    const int32_t dtype = small(&a, 1);
    const int64_t rows = whole(&a, 2), dim = whole(&a, 3), stride = whole(&a, 4);
    const void *tokens = pointer(&a, 5);
    const int32_t token_bytes = small(&a, 6);
    const int64_t count = whole(&a, 7), pad = whole(&a, 8);
    const float scale = (float)real(&a, 9);
    void *out = pointer(&a, 10);
    const int64_t out_stride = whole(&a, 11);
    uint64_t *bad = pointer(&a, 12);
    void *stream = pointer(&a, 13);
    CALL(lib.embed(table, dtype, rows, dim, stride, tokens, token_bytes, count, pad, scale, out,
                   out_stride, bad, stream));
}

static PyObject *embed_grad(PyObject *self, PyObject *const *at, Py_ssize_t n)
{
    args_t a;
    if (!begin(&a, at, n, 17, (void *)lib.embed_grad)) return NULL;
    const void *dy = pointer(&a, 0);
    const int32_t dtype = small(&a, 1);
    const int64_t stride = whole(&a, 2);
    const void *tokens = pointer(&a, 3);
    const int32_t token_bytes = small(&a, 4);
    const int64_t count = whole(&a, 5), pad = whole(&a, 6);
    const float scale = (float)real(&a, 7);
    void *grad = pointer(&a, 8);
    const int32_t grad_dtype = small(&a, 9);
    const int64_t rows = whole(&a, 10), dim = whole(&a, 11), grad_stride = whole(&a, 12);
    const int32_t accumulate = truth(&a, 13);
    void *workspace = pointer(&a, 14);
    const int64_t bytes = whole(&a, 15);
    void *stream = pointer(&a, 16);
    CALL(lib.embed_grad(dy, dtype, stride, tokens, token_bytes, count, pad, scale, grad,
                        grad_dtype, rows, dim, grad_stride, accumulate, workspace, bytes,
                        stream));
}

static PyObject *dropout(PyObject *self, PyObject *const *at, Py_ssize_t n)
{
    args_t a;
    if (!begin(&a, at, n, 10, (void *)lib.dropout)) return NULL;
    const void *x = pointer(&a, 0), *residual = pointer(&a, 1);
    void *out = pointer(&a, 2);
    const int32_t dtype = small(&a, 3);
    const int64_t count = whole(&a, 4);
    const double p = real(&a, 5);
    const uint64_t seed = word(&a, 6), offset = word(&a, 7);
    const int64_t first = whole(&a, 8);
    void *stream = pointer(&a, 9);
    CALL(lib.dropout(x, residual, out, dtype, count, p, seed, offset, first, stream));
}

static PyObject *quantize(PyObject *self, PyObject *const *at, Py_ssize_t n)
{
    args_t a;
    if (!begin(&a, at, n, 8, (void *)lib.quantize)) return NULL;
    const void *x = pointer(&a, 0);
    const int32_t dtype = small(&a, 1);
    const int64_t rows = whole(&a, 2), cols = whole(&a, 3), stride = whole(&a, 4);
    void *q = pointer(&a, 5), *qt = pointer(&a, 6), *stream = pointer(&a, 7);
    CALL(lib.quantize(x, dtype, rows, cols, stride, q, qt, stream));
}

static PyObject *dequantize(PyObject *self, PyObject *const *at, Py_ssize_t n)
{
    args_t a;
    if (!begin(&a, at, n, 7, (void *)lib.dequantize)) return NULL;
    const void *q = pointer(&a, 0);
    const int64_t rows = whole(&a, 1), cols = whole(&a, 2);
    void *out = pointer(&a, 3);
    const int32_t dtype = small(&a, 4);
    const int64_t stride = whole(&a, 5);
    void *stream = pointer(&a, 6);
    CALL(lib.dequantize(q, rows, cols, out, dtype, stride, stream));
}

static PyObject *matmul(PyObject *self, PyObject *const *at, Py_ssize_t n)
{
    args_t a;
    if (!begin(&a, at, n, 11, (void *)lib.matmul)) return NULL;
    const void *x = pointer(&a, 0);
    const int64_t m = whole(&a, 1);
    const void *y = pointer(&a, 2);
    const int64_t cols = whole(&a, 3), k = whole(&a, 4);
    const float alpha = (float)real(&a, 5);
    const int32_t accumulate = truth(&a, 6);
    void *out = pointer(&a, 7);
    const int32_t dtype = small(&a, 8);
    const int64_t stride = whole(&a, 9);
    void *stream = pointer(&a, 10);
    CALL(lib.matmul(x, m, y, cols, k, alpha, accumulate, out, dtype, stride, stream));
}

/* bind(embed, embed_grad, dropout, quantize, dequantize, matmul): addresses. */
static PyObject *bind(PyObject *self, PyObject *const *at, Py_ssize_t n)
{
    args_t a;
    if (!begin(&a, at, n, 6, (void *)&lib)) return NULL;
    void *p[6];
    for (int i = 0; i < 6; ++i) p[i] = pointer(&a, i);
    if (a.bad) return NULL;
    lib.embed = (__typeof__(lib.embed))p[0];
    lib.embed_grad = (__typeof__(lib.embed_grad))p[1];
    lib.dropout = (__typeof__(lib.dropout))p[2];
    lib.quantize = (__typeof__(lib.quantize))p[3];
    lib.dequantize = (__typeof__(lib.dequantize))p[4];
    lib.matmul = (__typeof__(lib.matmul))p[5];
    Py_RETURN_NONE;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}

static PyMethodDef methods[] = {METHOD(bind),     METHOD(embed),      METHOD(embed_grad),
                                METHOD(dropout),  METHOD(quantize),   METHOD(dequantize),
                                METHOD(matmul),   {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__calls(void)
{
    data_ptr_name = PyUnicode_InternFromString("data_ptr");
    return data_ptr_name ? PyModule_Create(&module) : NULL;
}
