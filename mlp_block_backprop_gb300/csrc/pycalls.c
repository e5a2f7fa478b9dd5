/* pycalls.c -- the latency-bound entry points of libmlpblk.so as CPython functions:
 * the calls of a serving step take microseconds on the device, and ctypes' argument
 * conversion is a large part of a call's host time (0.7 us on a Grace core; 0.15
 * here).  Each function takes the C function's arguments in order, addresses as
 * integers (None: NULL), and returns the MLPBLK_* code.  No checks but the argument
 * count: the Python classes and the library make them. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/mlpblk.h"

static void *ptr(PyObject *o) { return o == Py_None ? NULL : PyLong_AsVoidPtr(o); }

static int count(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return 1;
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", n, want);
    return 0;
}

/* Converts every argument before the call, so that a bad one calls nothing.  The call
 * runs without the interpreter's lock, as it does through ctypes: a launch can block (a
 * full launch queue, a kernel's first load), and what it waits for may be a callback that
 * needs the lock. */
#define CALL(name, N, ...)                                                       \
    static PyObject *py_##name(PyObject *self, PyObject *const *o, Py_ssize_t n) { \
        void *a[N];                                                              \
        (void)self;                                                              \
        if (!count(n, N)) return NULL;                                           \
        for (int i = 0; i < N; ++i) a[i] = ptr(o[i]);                            \
        if (PyErr_Occurred()) return NULL;                                       \
        int rc;                                                                  \
        Py_BEGIN_ALLOW_THREADS                                                   \
        rc = mlpblk_##name(__VA_ARGS__);                                         \
        Py_END_ALLOW_THREADS                                                     \
        return PyLong_FromLong(rc);                                              \
    }

CALL(moe_sort, 7, a[0], a[1], a[2], a[3], a[4], a[5], a[6])
CALL(moe_permute, 7, a[0], a[1], a[2], a[3], a[4], a[5], a[6])
CALL(moe_permute_backward, 5, a[0], a[1], a[2], a[3], a[4])
CALL(moe_unpermute, 7, a[0], a[1], a[2], a[3], a[4], a[5], a[6])
CALL(moe_unpermute_backward, 10, a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9])
CALL(fp4_quantize, 7, a[0], a[1], a[2], (int32_t)(intptr_t)a[3], a[4], a[5], a[6])
CALL(fp4_dequantize, 5, a[0], a[1], a[2], a[3], a[4])
CALL(fp4_matmul, 7, a[0], a[1], a[2], a[3], a[4], a[5], a[6])
CALL(fp4_matmul_grouped, 9, a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8])
CALL(fp4_wgrad_grouped, 8, a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7])

#define ENTRY(name) {"mlpblk_" #name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {
    ENTRY(moe_sort), ENTRY(moe_permute), ENTRY(moe_permute_backward), ENTRY(moe_unpermute),
    ENTRY(moe_unpermute_backward), ENTRY(fp4_quantize), ENTRY(fp4_dequantize), ENTRY(fp4_matmul),
    ENTRY(fp4_matmul_grouped), ENTRY(fp4_wgrad_grouped), {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mlpblk_calls", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__mlpblk_calls(void) { return PyModule_Create(&module); }
