/* binding.c -- Python calls of the entry points that a decode step makes many
 * times (4-bit products, cache, attention).  Small calls are bound by the host,
 * and ctypes takes 0.8 to 2.8 us to convert their 5 to 20 arguments (measured
 * per call; here 0.15 to 0.26).  Each function takes the C call's arguments as
 * integers (addresses too; None is NULL) and returns its status; the checks are
 * the Python side's and the library's.  The library is loaded by the Python
 * side, which hands over the addresses of its functions once (bind). */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "exl3.h"

static const char *const names[] = {"exl3_q4_gemm",     "exl3_kv_extend", "exl3_kv_write",       "exl3_kv_truncate",
                                    "exl3_kv_fork",     "exl3_kv_compact", "exl3_paged_attention"};
enum { Q4_GEMM, KV_EXTEND, KV_WRITE, KV_TRUNCATE, KV_FORK, KV_COMPACT, ATTENTION, COUNT };
static void *entry[COUNT];

static void *ptr(PyObject *o)
{
    return o == Py_None ? NULL : (void *)(size_t)PyLong_AsUnsignedLongLong(o);
}
static long long wide(PyObject *o)
{
    return PyLong_AsLongLong(o);
}
static int num(PyObject *o)
{
    const long v = PyLong_AsLong(o);
    if (v != (int)v && !PyErr_Occurred()) PyErr_SetString(PyExc_OverflowError, "argument does not fit a C int");
    return (int)v;
}

#define FUNCTION(name) static PyObject *name(PyObject *self, PyObject *const *o, Py_ssize_t count)

/* Whether there are as many arguments as there should be; sets the error. */
static int expect(int which, Py_ssize_t have, Py_ssize_t want)
{
    if (entry[which] && have == want) return 1;
    PyErr_Format(PyExc_TypeError, "%s: takes %zd arguments, got %zd", names[which], want, have);
    return 0;
}

#define RETURN_CALL(call)               \
    do {                                \
        int status;                     \
        if (PyErr_Occurred()) return NULL; \
        Py_BEGIN_ALLOW_THREADS          \
        status = call;                  \
        Py_END_ALLOW_THREADS            \
        return PyLong_FromLong(status); \
    } while (0)

FUNCTION(q4_gemm)
{
    if (!expect(Q4_GEMM, count, 13)) return NULL;
    const int m = num(o[0]), fp32 = num(o[6]), k_in = num(o[7]), n_out = num(o[8]), group = num(o[9]);
    const uint16_t *x = ptr(o[1]), *scale = ptr(o[3]);
    const uint32_t *packed = ptr(o[2]);
    const uint8_t *zero = ptr(o[4]);
    void *y = ptr(o[5]), *ws = ptr(o[10]), *stream = ptr(o[12]);
    const size_t room = (size_t)wide(o[11]);
    RETURN_CALL(((__typeof__(&exl3_q4_gemm))entry[Q4_GEMM])(m, x, packed, scale, zero, y, fp32, k_in, n_out, group, ws, room, stream));
}

FUNCTION(kv_extend)
{
    if (!expect(KV_EXTEND, count, 6)) return NULL;
    const exl3_kv_cache_t *cache = ptr(o[0]);
    const int n = num(o[1]), m = num(o[2]);
    const int32_t *seqs = ptr(o[3]), *counts = ptr(o[4]);
    void *stream = ptr(o[5]);
    RETURN_CALL(((__typeof__(&exl3_kv_extend))entry[KV_EXTEND])(cache, n, m, seqs, counts, stream));
}

FUNCTION(kv_write)
{
    if (!expect(KV_WRITE, count, 11)) return NULL;
    const exl3_kv_cache_t *cache = ptr(o[0]);
    const int layer = num(o[1]), n = num(o[2]), m = num(o[3]);
    const int32_t *seqs = ptr(o[4]), *counts = ptr(o[5]);
    const uint16_t *k = ptr(o[6]), *v = ptr(o[7]);
    const long long bs = wide(o[8]), rs = wide(o[9]);
    void *stream = ptr(o[10]);
    RETURN_CALL(((__typeof__(&exl3_kv_write))entry[KV_WRITE])(cache, layer, n, m, seqs, counts, k, v, bs, rs, stream));
}

/* truncate, fork: a cache, n, two lists, a stream */
static PyObject *two_lists(int which, PyObject *const *o, Py_ssize_t count)
{
    if (!expect(which, count, 5)) return NULL;
    const exl3_kv_cache_t *cache = ptr(o[0]);
    const int n = num(o[1]);
    const int32_t *one = ptr(o[2]), *other = ptr(o[3]);
    void *stream = ptr(o[4]);
    RETURN_CALL(((__typeof__(&exl3_kv_fork))entry[which])(cache, n, one, other, stream));
}
FUNCTION(kv_truncate) { return two_lists(KV_TRUNCATE, o, count); }
FUNCTION(kv_fork) { return two_lists(KV_FORK, o, count); }

FUNCTION(kv_compact)
{
    if (!expect(KV_COMPACT, count, 2)) return NULL;
    const exl3_kv_cache_t *cache = ptr(o[0]);
    void *stream = ptr(o[1]);
    RETURN_CALL(((__typeof__(&exl3_kv_compact))entry[KV_COMPACT])(cache, stream));
}

FUNCTION(paged_attention)
{
    if (!expect(ATTENTION, count, 20)) return NULL;
    const exl3_kv_cache_t *cache = ptr(o[0]);
    const int layer = num(o[1]), n = num(o[2]), m = num(o[3]), heads = num(o[9]), window = num(o[11]), sinks = num(o[12]);
    const int32_t *seqs = ptr(o[4]), *counts = ptr(o[5]);
    const uint16_t *q = ptr(o[6]);
    const long long qb = wide(o[7]), qr = wide(o[8]), ob = wide(o[14]), orow = wide(o[15]);
    const float scale = (float)PyFloat_AsDouble(o[10]);
    uint16_t *out = ptr(o[13]);
    float *lse = ptr(o[16]);
    void *ws = ptr(o[17]), *stream = ptr(o[19]);
    const size_t room = (size_t)wide(o[18]);
    RETURN_CALL(((__typeof__(&exl3_paged_attention))entry[ATTENTION])(cache, layer, n, m, seqs, counts, q, qb, qr, heads, scale, window,
                                                                     sinks, out, ob, orow, lse, ws, room, stream));
}

/* bind(addresses): of the functions in `names`, in that order */
static PyObject *bind(PyObject *self, PyObject *addresses)
{
    void *found[COUNT];
    for (int i = 0; i < COUNT; ++i) {
        PyObject *item = PySequence_GetItem(addresses, i);
        if (!item) return NULL;
        found[i] = ptr(item);
        Py_DECREF(item);
    }
    if (PyErr_Occurred()) return NULL;
    for (int i = 0; i < COUNT; ++i) entry[i] = found[i];
    Py_RETURN_NONE;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {METHOD(q4_gemm), METHOD(kv_extend),  METHOD(kv_write),        METHOD(kv_truncate),
                                METHOD(kv_fork), METHOD(kv_compact), METHOD(paged_attention), {"bind", bind, METH_O, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void)
{
    PyObject *m = PyModule_Create(&module);
    if (!m) return NULL;
    PyObject *list = PyTuple_New(COUNT);
    for (int i = 0; list && i < COUNT; ++i) PyTuple_SET_ITEM(list, i, PyUnicode_FromString(names[i]));
    if (!list || PyModule_AddObject(m, "NAMES", list) < 0) return NULL;
    return m;
}
