/*
 * CPython module between expert_ops.py and the entry points of expert_ops.h:
 * one function an entry point, integers (None: a NULL pointer) in the order of
 * the C arguments, the status or size back.  A call through ctypes costs 4 to
 * 5 us, which is what a small kernel takes; this costs a tenth of it.  The
 * library is already loaded: bind() takes the entry points' addresses.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "expert_ops.h"

enum { LINEAR, WEIGHT_GRAD, QUANTIZE, DEQUANTIZE, MX4_SPACE, MX4_LINEAR, ROUTE_SPACE, ROUTE, ROUTE_GRAD, COUNT };

static const char *const names[COUNT] = {
    "expert_grouped_linear", "expert_grouped_weight_grad", "expert_mx4_quantize",   "expert_mx4_dequantize",
    "expert_mx4_workspace",  "expert_mx4_linear",          "expert_route_workspace", "expert_route",
    "expert_route_grad"};
static void *entry[COUNT];

#define MOST_ARGS 17

/* The arguments as integers; -1 and an exception where one is none. */
static int integers(int which, PyObject *const *args, Py_ssize_t n, Py_ssize_t want, int64_t *v)
{
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%s takes %zd arguments (%zd given)", names[which], want, n);
        return -1;
    }
    if (!entry[which]) {
        PyErr_Format(PyExc_RuntimeError, "%s is not bound", names[which]);
        return -1;
    }
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (args[i] == Py_None) {
            v[i] = 0;
        } else {
            v[i] = PyLong_AsLongLong(args[i]);
            if (v[i] == -1 && PyErr_Occurred()) {
                /* An address with the top bit set. */
                if (!PyErr_ExceptionMatches(PyExc_OverflowError)) return -1;
                PyErr_Clear();
                v[i] = (int64_t)PyLong_AsUnsignedLongLong(args[i]);
                if (PyErr_Occurred()) return -1;
            }
        }
    }
    return 0;
}

/* An int argument: a value outside an int is outside every range they have. */
static int small(int64_t v) { return v < -1 || v > 0x7fffffff ? -1 : (int)v; }

#define P(i) ((void *)(intptr_t)v[i])
#define CALL(which, want, type, expression)                                                       \
    int64_t v[MOST_ARGS];                                                                         \
    long long result;                                                                             \
    if (integers(which, args, n, want, v) < 0) return NULL;                                       \
    Py_BEGIN_ALLOW_THREADS result = ((type)entry[which]) expression;                              \
    Py_END_ALLOW_THREADS return PyLong_FromLongLong(result)

typedef int (*linear_t)(int, int64_t, int64_t, int64_t, int64_t, const void *, int64_t, const void *, int, int64_t,
                        int64_t, const int *, const float *, int, void *, int64_t, void *);
static PyObject *linear(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    CALL(LINEAR, 17, linear_t, (small(v[0]), v[1], v[2], v[3], v[4], P(5), v[6], P(7), small(v[8]), v[9], v[10], P(11),
                                P(12), small(v[13]), P(14), v[15], P(16)));
}

typedef int (*weight_grad_t)(int, int64_t, int64_t, int64_t, int64_t, const void *, int64_t, const void *, int64_t,
                             const int *, void *, int64_t, int64_t, void *);
static PyObject *weight_grad(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    CALL(WEIGHT_GRAD, 14, weight_grad_t,
         (small(v[0]), v[1], v[2], v[3], v[4], P(5), v[6], P(7), v[8], P(9), P(10), v[11], v[12], P(13)));
}

typedef int (*quantize_t)(int, int64_t, int64_t, const void *, int, int64_t, void *, void *, void *);
static PyObject *quantize(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    CALL(QUANTIZE, 9, quantize_t, (small(v[0]), v[1], v[2], P(3), small(v[4]), v[5], P(6), P(7), P(8)));
}

typedef int (*dequantize_t)(int, int64_t, int64_t, const void *, const void *, void *, int64_t, void *);
static PyObject *dequantize(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    CALL(DEQUANTIZE, 8, dequantize_t, (small(v[0]), v[1], v[2], P(3), P(4), P(5), v[6], P(7)));
}

typedef int64_t (*mx4_space_t)(int64_t, int64_t, int64_t, int64_t);
static PyObject *mx4_space(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    CALL(MX4_SPACE, 4, mx4_space_t, (v[0], v[1], v[2], v[3]));
}

typedef int (*mx4_linear_t)(int, int64_t, int64_t, int64_t, int64_t, const void *, int64_t, const void *, const void *,
                            const int *, const float *, int, void *, int64_t, void *, int64_t, void *);
static PyObject *mx4_linear(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    CALL(MX4_LINEAR, 17, mx4_linear_t, (small(v[0]), v[1], v[2], v[3], v[4], P(5), v[6], P(7), P(8), P(9), P(10),
                                        small(v[11]), P(12), v[13], P(14), v[15], P(16)));
}

typedef int64_t (*route_space_t)(int64_t, int64_t);
static PyObject *route_space(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    CALL(ROUTE_SPACE, 2, route_space_t, (v[0], v[1]));
}

typedef int (*route_t)(int, int64_t, int64_t, int64_t, int, const void *, int64_t, float *, int *, int *, int *, void *,
                       int64_t, void *);
static PyObject *route(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    CALL(ROUTE, 14, route_t, (small(v[0]), v[1], v[2], v[3], small(v[4]), P(5), v[6], P(7), P(8), P(9), P(10), P(11),
                              v[12], P(13)));
}

typedef int (*route_grad_t)(int, int64_t, int64_t, int64_t, int, const void *, int64_t, const float *, const int *,
                            const float *, void *, int64_t, void *);
static PyObject *route_grad(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    CALL(ROUTE_GRAD, 13, route_grad_t, (small(v[0]), v[1], v[2], v[3], small(v[4]), P(5), v[6], P(7), P(8), P(9), P(10),
                                        v[11], P(12)));
}

static PyObject *bind(PyObject *self, PyObject *addresses)
{
    for (int i = 0; i < COUNT; ++i) {
        PyObject *a = PyMapping_GetItemString(addresses, names[i]);
        if (!a) return NULL;
        entry[i] = PyLong_AsVoidPtr(a);
        Py_DECREF(a);
        if (PyErr_Occurred()) return NULL;
    }
    Py_RETURN_NONE;
}

#define FAST(name, f) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {
    {"bind", bind, METH_O, "bind({name: address}) for every entry point of expert_ops.h"},
    FAST("expert_grouped_linear", linear),
    FAST("expert_grouped_weight_grad", weight_grad),
    FAST("expert_mx4_quantize", quantize),
    FAST("expert_mx4_dequantize", dequantize),
    FAST("expert_mx4_workspace", mx4_space),
    FAST("expert_mx4_linear", mx4_linear),
    FAST("expert_route_workspace", route_space),
    FAST("expert_route", route),
    FAST("expert_route_grad", route_grad),
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_expert_binding",
                                    "The entry points of expert_ops.h, on integers.", -1, methods};

PyMODINIT_FUNC PyInit__expert_binding(void) { return PyModule_Create(&module); }
