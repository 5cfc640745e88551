/* pyargs.h -- conversions of the CPython modules that call the libraries
 * without ctypes, which they follow: integers with __index__, floats rounded
 * once to binary32, pointers from an int, None (NULL) or an object with an int
 * `value`. */
#ifndef OU_PYARGS_H
#define OU_PYARGS_H

#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>
#include <string.h>

static int to_i64(PyObject* o, long long* out)
{
    *out = PyLong_AsLongLong(o);
    return !(*out == -1 && PyErr_Occurred());
}

static inline int to_i32(PyObject* o, int* out)
{
    long long v;
    if (!to_i64(o, &v)) return 0;
    *out = (int)v;
    return 1;
}

static int to_f32(PyObject* o, float* out)
{
    const double d = PyFloat_AsDouble(o);
    if (d == -1.0 && PyErr_Occurred()) return 0;
    *out = (float)d;
    return 1;
}

static int to_ptr(PyObject* o, void** out)
{
    if (o == Py_None) {
        *out = NULL;
        return 1;
    }
    if (PyLong_Check(o)) {
        const unsigned long long v = PyLong_AsUnsignedLongLong(o);
        if (v == (unsigned long long)-1 && PyErr_Occurred()) return 0;
        *out = (void*)(uintptr_t)v;
        return 1;
    }
    PyObject* v = PyObject_GetAttrString(o, "value");   /* c_void_p */
    if (!v) return 0;
    const int ok = to_ptr(v, out);
    Py_DECREF(v);
    return ok;
}

static int nargs_ok(const char* name, Py_ssize_t got, Py_ssize_t want)
{
    if (got == want) return 1;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments (%zd given)", name, want, got);
    return 0;
}

#endif
