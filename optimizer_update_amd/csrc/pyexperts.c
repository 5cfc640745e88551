/* pyexperts.c -- CPython entry points of liboptimizer_experts.so: the same C
 * functions that the ctypes binding calls, with the same positional arguments,
 * converted here.  A call's arguments are 6 to 18 numbers, whose conversion by
 * ctypes is a good part of the host cost of a small call.  Every check stays in
 * the library; the calls run with the GIL released, as ctypes' do.
 */
#include "pyargs.h"

#include "../../include/optimizer_experts.h"

typedef union {
    int i;
    long long l;
    float f;
    void* p;
} arg;

/* An int that is none would be another number (2^32 + 1 experts: one). */
static int to_int(const char* name, Py_ssize_t at, PyObject* o, int* out)
{
    long long v;
    if (!to_i64(o, &v)) return 0;
    if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_Format(PyExc_OverflowError, "%s: argument %zd does not fit 32 bits", name, at + 1);
        return 0;
    }
    *out = (int)v;
    return 1;
}

/* kinds: a letter an argument, i int, l int64, f binary32, p pointer */
static int convert(const char* name, const char* kinds, PyObject* const* a, Py_ssize_t na, arg* out)
{
    if (!nargs_ok(name, na, (Py_ssize_t)strlen(kinds))) return 0;
    for (Py_ssize_t k = 0; k < na; ++k) {
        int ok = 0;
        switch (kinds[k]) {
        case 'i': ok = to_int(name, k, a[k], &out[k].i); break;
        case 'l': ok = to_i64(a[k], &out[k].l); break;
        case 'f': ok = to_f32(a[k], &out[k].f); break;
        case 'p': ok = to_ptr(a[k], &out[k].p); break;
        }
        if (!ok) return 0;
    }
    return 1;
}

#define ENTRY(name, kinds, call)                                                                  \
    static PyObject* py_##name(PyObject* self, PyObject* const* a, Py_ssize_t na)                 \
    {                                                                                             \
        arg v[sizeof(kinds)];                                                                     \
        int st;                                                                                   \
        (void)self;                                                                               \
        if (!convert(#name, kinds, a, na, v)) return NULL;                                        \
        Py_BEGIN_ALLOW_THREADS st = call;                                                         \
        Py_END_ALLOW_THREADS return PyLong_FromLong(st);                                          \
    }

ENTRY(ou_route_topk, "iplilipiiiifpippp",
      ou_route_topk(v[0].i, v[1].p, v[2].l, v[3].i, v[4].l, v[5].i, v[6].p, v[7].i, v[8].i, v[9].i, v[10].i, v[11].f,
                    v[12].p, v[13].i, v[14].p, v[15].p, v[16].p))
ENTRY(ou_route_topk_backward, "ipliliifppipp",
      ou_route_topk_backward(v[0].i, v[1].p, v[2].l, v[3].i, v[4].l, v[5].i, v[6].i, v[7].f, v[8].p, v[9].p, v[10].i,
                             v[11].p, v[12].p))
ENTRY(ou_route_order, "plipppplp",
      ou_route_order(v[0].p, v[1].l, v[2].i, v[3].p, v[4].p, v[5].p, v[6].p, v[7].l, v[8].p))
ENTRY(ou_route_dispatch, "iplllippplip",
      ou_route_dispatch(v[0].i, v[1].p, v[2].l, v[3].l, v[4].l, v[5].i, v[6].p, v[7].p, v[8].p, v[9].l, v[10].i, v[11].p))
ENTRY(ou_route_combine, "iplllippplplp",
      ou_route_combine(v[0].i, v[1].p, v[2].l, v[3].l, v[4].l, v[5].i, v[6].p, v[7].p, v[8].p, v[9].l, v[10].p, v[11].l,
                       v[12].p))
ENTRY(ou_route_combine_backward, "ipllliplpppppp",
      ou_route_combine_backward(v[0].i, v[1].p, v[2].l, v[3].l, v[4].l, v[5].i, v[6].p, v[7].l, v[8].p, v[9].p, v[10].p,
                                v[11].p, v[12].p, v[13].p))
ENTRY(ou_route_balance, "ppifpp", ou_route_balance(v[0].p, v[1].p, v[2].i, v[3].f, v[4].p, v[5].p))
ENTRY(ou_int4_matmul, "ipllipipplliplp",
      ou_int4_matmul(v[0].i, v[1].p, v[2].l, v[3].l, v[4].i, v[5].p, v[6].i, v[7].p, v[8].p, v[9].l, v[10].l, v[11].i,
                     v[12].p, v[13].l, v[14].p))
ENTRY(ou_int4_grouped_matmul, "ipllipippllipiplip",
      ou_int4_grouped_matmul(v[0].i, v[1].p, v[2].l, v[3].l, v[4].i, v[5].p, v[6].i, v[7].p, v[8].p, v[9].l, v[10].l,
                             v[11].i, v[12].p, v[13].i, v[14].p, v[15].l, v[16].i, v[17].p))

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, NULL}

static PyMethodDef methods[] = {
    METHOD(ou_route_topk),    METHOD(ou_route_topk_backward),    METHOD(ou_route_order),   METHOD(ou_route_dispatch),
    METHOD(ou_route_combine), METHOD(ou_route_combine_backward), METHOD(ou_route_balance), METHOD(ou_int4_matmul),
    METHOD(ou_int4_grouped_matmul), {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast_experts", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fast_experts(void) { return PyModule_Create(&module); }
