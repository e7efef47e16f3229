/* What the modules that marshal arguments share: conversions of a call's arguments,
 * an entry point as a Python function, the module itself. */
#pragma once

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
#define F(i) const float f##i = (float)PyFloat_AsDouble(a[i])
#define S(i) void *s = stream(a[i])

static PyObject *py_set_current_stream(PyObject *self, PyObject *f)
{
    (void)self;
    Py_INCREF(f);
    Py_XSETREF(current_stream, f);
    Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, NULL}
#define BINDING_END \
    {"set_current_stream", py_set_current_stream, METH_O, "The callable that gives the stream of a call with None."}, \
    {NULL, NULL, 0, NULL}

/* The module of that name, its functions in `methods`. */
#define BINDING_MODULE(name)                                                  \
    static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, #name, NULL, -1, methods, NULL, NULL, NULL, NULL}; \
    PyMODINIT_FUNC PyInit_##name(void)                                        \
    {                                                                         \
        s_data_ptr = PyUnicode_InternFromString("data_ptr");                  \
        s_cuda_stream = PyUnicode_InternFromString("cuda_stream");            \
        Py_INCREF(Py_None);                                                   \
        current_stream = Py_None;                                             \
        if (!s_data_ptr || !s_cuda_stream) return NULL;                       \
        return PyModule_Create(&module);                                      \
    }
