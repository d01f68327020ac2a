/* binding.c — CPython entry to the expert-MLP functions of the C ABI.
 *
 * The operators take a few microseconds on the GPU and up to nineteen
 * arguments; converting those through ctypes takes 1.7 us a call, through
 * this module 0.3.  Arguments are marshalled and nothing else: pointers come
 * as tensors, ints or None (NULL), the result is the status.  The last argument
 * is the device whose memory the call works on: where a tensor is on another,
 * or on the host, the C function is not called and the result is -1.  (The
 * check takes 0.1 to 0.2 us of a call's 3.8 to 5.6.)  The interpreter lock is
 * released around the call, as ctypes does. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "swiglu_mlp.h"

static PyObject *get_device, *data_ptr;       /* names of a tensor's methods */

static void *pointer(PyObject *o, long device, int *elsewhere)
{
    if (o == Py_None) return NULL;
    if (PyLong_Check(o)) return PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) return NULL;         /* an argument before this one */
    PyObject *on = PyObject_CallMethodObjArgs(o, get_device, NULL);
    if (on == NULL) return NULL;
    if (PyLong_AsLong(on) != device) *elsewhere = 1;
    Py_DECREF(on);
    PyObject *at = PyObject_CallMethodObjArgs(o, data_ptr, NULL);
    if (at == NULL) return NULL;
    void *p = PyLong_AsVoidPtr(at);
    Py_DECREF(at);
    return p;
}
static int64_t whole(PyObject *o) { return PyLong_AsLongLong(o); }
static float real(PyObject *o) { return (float)PyFloat_AsDouble(o); }

#define P(i) pointer(a[i], device, &elsewhere)
#define I(i) whole(a[i])
#define F(i) real(a[i])

/* A Python function `name` of `count` arguments and the device: ENTRY, their
 * conversion into locals, then CALL of the C function with those. */
#define ENTRY(name, count)                                                                       \
    static PyObject *py_##name(PyObject *self, PyObject *const *a, Py_ssize_t n)                 \
    {                                                                                            \
        (void)self;                                                                              \
        if (n != count + 1) {                                                                    \
            PyErr_SetString(PyExc_TypeError, #name " takes " #count " arguments and the device"); \
            return NULL;                                                                         \
        }                                                                                        \
        const long device = PyLong_AsLong(a[count]);                                             \
        int elsewhere = 0;
#define CALL(...)                                                                                \
        if (PyErr_Occurred()) return NULL;                                                       \
        if (elsewhere) return PyLong_FromLong(-1);                                               \
        int rc;                                                                                  \
        Py_BEGIN_ALLOW_THREADS;                                                                  \
        rc = __VA_ARGS__;                                                                        \
        Py_END_ALLOW_THREADS;                                                                    \
        return PyLong_FromLong(rc);                                                              \
    }

ENTRY(gemm_grouped, 17)
    int tB = (int)I(0); int64_t G = I(1), M = I(2), N = I(3), K = I(4); float alpha = F(5);
    void *A = P(6); int64_t lda = I(7); void *B = P(8); int64_t ldb = I(9), sB = I(10);
    void *off = P(11); float beta = F(12); void *C = P(13); int64_t ldc = I(14);
    int dt = (int)I(15); void *st = P(16);
    CALL(gemm_grouped(tB, G, M, N, K, alpha, A, lda, B, ldb, sB, off, beta, C, ldc, dt, st))

ENTRY(gemm_grouped_wgrad, 16)
    int64_t G = I(0), M = I(1), N = I(2), K = I(3); float alpha = F(4);
    void *A = P(5); int64_t lda = I(6); void *D = P(7); int64_t ldd = I(8); void *off = P(9);
    float beta = F(10); void *C = P(11); int64_t ldc = I(12), sC = I(13); int dt = (int)I(14);
    void *st = P(15);
    CALL(gemm_grouped_wgrad(G, M, N, K, alpha, A, lda, D, ldd, off, beta, C, ldc, sC, dt, st))

ENTRY(swiglu_grouped, 9)
    void *A = P(0), *W = P(1), *Y = P(2), *off = P(3);
    int64_t G = I(4), M = I(5), N = I(6), K = I(7); void *st = P(8);
    CALL(swiglu_grouped(A, W, Y, off, G, M, N, K, st))

ENTRY(swiglu_grouped_grad, 11)
    void *A = P(0), *W = P(1), *dY = P(2), *Y = P(3), *dH = P(4), *off = P(5);
    int64_t G = I(6), M = I(7), N = I(8), K = I(9); void *st = P(10);
    CALL(swiglu_grouped_grad(A, W, dY, Y, dH, off, G, M, N, K, st))

ENTRY(mx4_quantize, 13)
    int f = (int)I(0); int64_t G = I(1), M = I(2), K = I(3); void *X = P(4); int64_t ldx = I(5);
    int type = (int)I(6); float scale = F(7); void *off = P(8), *Q = P(9); int64_t ldq = I(10);
    void *S = P(11), *st = P(12);
    CALL(mx4_quantize(f, G, M, K, X, ldx, type, scale, off, Q, ldq, S, st))

ENTRY(mx4_dequantize, 13)
    int f = (int)I(0); int64_t G = I(1), M = I(2), K = I(3); void *Q = P(4); int64_t ldq = I(5);
    void *S = P(6); float scale = F(7); void *off = P(8), *X = P(9); int64_t ldx = I(10);
    int type = (int)I(11); void *st = P(12);
    CALL(mx4_dequantize(f, G, M, K, Q, ldq, S, scale, off, X, ldx, type, st))

ENTRY(gemm_mx4, 19)
    int f = (int)I(0); int64_t G = I(1), M = I(2), N = I(3), K = I(4); float alpha = F(5);
    void *A = P(6); int64_t lda = I(7); void *SA = P(8), *B = P(9);
    int64_t ldb = I(10), sB = I(11); void *SB = P(12), *off = P(13); float beta = F(14);
    void *C = P(15); int64_t ldc = I(16); int type = (int)I(17); void *st = P(18);
    CALL(gemm_mx4(f, G, M, N, K, alpha, A, lda, SA, B, ldb, sB, SB, off, beta, C, ldc, type, st))

ENTRY(swiglu_mx4, 13)
    int f = (int)I(0); void *A = P(1), *SA = P(2), *W = P(3), *SW = P(4), *Y = P(5), *off = P(6);
    int64_t G = I(7), M = I(8), N = I(9), K = I(10); float alpha = F(11); void *st = P(12);
    CALL(swiglu_mx4(f, A, SA, W, SW, Y, off, G, M, N, K, alpha, st))

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {
    METHOD(gemm_grouped), METHOD(gemm_grouped_wgrad), METHOD(swiglu_grouped),
    METHOD(swiglu_grouped_grad), METHOD(mx4_quantize), METHOD(mx4_dequantize), METHOD(gemm_mx4),
    METHOD(swiglu_mx4), {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void)
{
    get_device = PyUnicode_InternFromString("get_device");
    data_ptr = PyUnicode_InternFromString("data_ptr");
    return get_device != NULL && data_ptr != NULL ? PyModule_Create(&module) : NULL;
}
