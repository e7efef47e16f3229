/* Argument marshalling of the many-token and 8-bit calls, as a CPython module.
 *
 * Each function takes the C entry point's arguments (a tensor, an address or
 * None where it takes a pointer; a stream object, a handle or None, torch's
 * current stream, where it takes a stream) and returns its status.  A call
 * of a small batch is bound by the host: converting eight arguments here costs
 * about 0.3 us where the ctypes route costs 1.2.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "smoe.h"

static PyObject *s_data_ptr, *s_cuda_stream, *current_stream;

/* A device address: None, an int, or an object with data_ptr(). */
static void *pointer(PyObject *o)
{
    if (o == Py_None) return NULL;
    if (PyLong_Check(o)) return PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) return NULL;  /* an earlier argument's */
    PyObject *v = PyObject_CallMethodNoArgs(o, s_data_ptr);
    if (!v) return NULL;
    void *p = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return p;
}

static int integer(PyObject *o)
{
    const long v = PyLong_AsLong(o);
    if (v == (long)(int)v) return (int)v;
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_OverflowError, "an argument does not fit 32 bits");
    return 0;
}

static void *stream(PyObject *o)
{
    if (PyLong_Check(o)) return PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) return NULL;
    PyObject *v = o == Py_None ? PyObject_CallNoArgs(current_stream) : PyObject_GetAttr(o, s_cuda_stream);
    if (!v) return NULL;
    void *p = v == Py_None ? NULL : PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return p;
}

static PyObject *arity(const char *name, Py_ssize_t want, Py_ssize_t got)
{
    return PyErr_Format(PyExc_TypeError, "%s takes %zd arguments (%zd given)", name, want, got);
}

/* The entry point with the converted arguments, the interpreter released as
 * around any call that may wait (a launch into a full queue). */
#define ENTRY(name, count, convert, call)                                     \
    static PyObject *py_##name(PyObject *self, PyObject *const *a, Py_ssize_t n) \
    {                                                                         \
        (void)self;                                                           \
        if (n != count) return arity(#name, count, n);                        \
        convert;                                                              \
        if (PyErr_Occurred()) return NULL;                                    \
        int status;                                                           \
        Py_BEGIN_ALLOW_THREADS                                                \
        status = name call;                                                   \
        Py_END_ALLOW_THREADS                                                  \
        return PyLong_FromLong(status);                                       \
    }

#define P(i) void *p##i = pointer(a[i])
#define I(i) const int v##i = integer(a[i])
#define Z(i) const size_t z##i = PyLong_AsSize_t(a[i])
#define S(i) void *s = stream(a[i])

ENTRY(smoe_topk_rows, 8, P(0); I(1); I(2); I(3); I(4); P(5); P(6); S(7), (p0, v1, v2, v3, v4, p5, p6, s))
ENTRY(smoe_topk_rows_backward, 8, P(0); P(1); P(2); I(3); I(4); I(5); P(6); S(7), (p0, p1, p2, v3, v4, v5, p6, s))
ENTRY(smoe_dispatch_tokens, 14, P(0); I(1); I(2); I(3); P(4); I(5); I(6); P(7); P(8); P(9); P(10); P(11); Z(12); S(13),
      (p0, v1, v2, v3, p4, v5, v6, p7, p8, p9, p10, p11, z12, s))
ENTRY(smoe_dispatch_tokens_backward, 8, P(0); I(1); P(2); I(3); I(4); I(5); P(6); S(7), (p0, v1, p2, v3, v4, v5, p6, s))
ENTRY(smoe_combine_tokens, 9, P(0); I(1); P(2); P(3); I(4); I(5); I(6); P(7); S(8), (p0, v1, p2, p3, v4, v5, v6, p7, s))
ENTRY(smoe_combine_tokens_backward, 11, P(0); P(1); I(2); P(3); P(4); I(5); I(6); I(7); P(8); P(9); S(10),
      (p0, p1, v2, p3, p4, v5, v6, v7, p8, p9, s))
ENTRY(smoe_quantize_rows_q8, 8, P(0); I(1); I(2); I(3); I(4); P(5); P(6); S(7), (p0, v1, v2, v3, v4, p5, p6, s))
ENTRY(smoe_matmul_q8, 12, P(0); P(1); I(2); P(3); P(4); I(5); I(6); P(7); I(8); P(9); Z(10); S(11),
      (p0, p1, v2, p3, p4, v5, v6, p7, v8, p9, z10, s))
ENTRY(smoe_experts_matmul_q8, 17,
      P(0); P(1); I(2); P(3); I(4); P(5); I(6); I(7); P(8); P(9); I(10); I(11); P(12); I(13); P(14); Z(15); S(16),
      (p0, p1, v2, p3, v4, p5, v6, v7, p8, p9, v10, v11, p12, v13, p14, z15, s))

static PyObject *py_set_current_stream(PyObject *self, PyObject *f)
{
    (void)self;
    Py_INCREF(f);
    Py_XSETREF(current_stream, f);
    Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {
    FAST(smoe_topk_rows),
    FAST(smoe_topk_rows_backward),
    FAST(smoe_dispatch_tokens),
    FAST(smoe_dispatch_tokens_backward),
    FAST(smoe_combine_tokens),
    FAST(smoe_combine_tokens_backward),
    FAST(smoe_quantize_rows_q8),
    FAST(smoe_matmul_q8),
    FAST(smoe_experts_matmul_q8),
    {"set_current_stream", py_set_current_stream, METH_O, "The callable that gives the stream of a call with None."},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void)
{
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    Py_INCREF(Py_None);
    current_stream = Py_None;
    if (!s_data_ptr || !s_cuda_stream) return NULL;
    return PyModule_Create(&module);
}
