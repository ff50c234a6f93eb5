/* py_calls.c -- argument marshalling of the decode-step calls for Python.
 *
 * The binding forwards to libwq through ctypes; for the calls that a decode loop makes once
 * per layer and token, converting up to 25 arguments there takes longer than the kernels run
 * (wq_kv_append of 64 tokens: 7.3 us of host time through ctypes, 2.3 us on the GPU).  This
 * module converts them with the C API and calls the same entry points, whose addresses the
 * binding passes in; it checks types and nothing else. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <limits.h>
#include <stdint.h>

#include "../../include/wq.h"

static wq_status (*f_rope)(int, int, int, int, unsigned, const float *, int64_t, const int32_t *,
                           const float *, int, float *, int64_t, wq_stream_t);
static wq_status (*f_append)(const wq_kv_cache *, int, int, int, unsigned, const float *, int64_t,
                             const float *, int64_t, const float *, int64_t, const int32_t *,
                             const float *, int, int, const int32_t *, const int32_t *,
                             const int32_t *, int, float *, int64_t, float *, int32_t *, int64_t,
                             wq_stream_t);
static wq_status (*f_attn)(const wq_kv_cache *, int, int, float, int, const float *, int64_t,
                           const int32_t *, int, const int32_t *, const float *, int64_t, float *,
                           int64_t, float *, const float *, float *, int64_t, void *, size_t,
                           wq_stream_t);
static wq_status (*f_evict)(const wq_kv_cache *, int, const int32_t *, int, const int32_t *,
                            const int32_t *, int, int, int, const float *, const int32_t *,
                            float *, int32_t *, int64_t, int32_t *, void *, size_t, wq_stream_t);
static PyObject *current_stream; /* () -> int */
static PyObject *cache_type;     /* KvCache */
static PyObject *s_data_ptr, *s_cuda_stream;

/* Each converter returns one argument; on failure it sets an exception and counts.  After a
 * failure the others return at once: no Python may run with an exception set. */
static long long as_i64(PyObject *o, int *bad) {
    if (*bad) return 0;
    if (PyLong_Check(o)) {
        const long long v = PyLong_AsLongLong(o);
        if (v == -1 && PyErr_Occurred()) ++*bad;
        return v;
    }
    PyObject *i = PyNumber_Index(o); /* numpy integers */
    if (!i) {
        ++*bad;
        return 0;
    }
    const long long v = PyLong_AsLongLong(i);
    Py_DECREF(i);
    if (v == -1 && PyErr_Occurred()) ++*bad;
    return v;
}

static int as_int(PyObject *o, int *bad) {
    const long long v = as_i64(o, bad);
    if (!*bad && (v < INT_MIN || v > (long long)UINT_MAX)) {
        PyErr_SetString(PyExc_OverflowError, "argument does not fit a C int");
        ++*bad;
    }
    return (int)v;
}

static float as_float(PyObject *o, int *bad) {
    if (*bad) return 0.f;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) ++*bad;
    return (float)v;
}

/* None, an address, or an object with data_ptr() (a tensor). */
static void *as_ptr(PyObject *o, int *bad) {
    if (*bad || o == Py_None) return NULL;
    if (PyLong_Check(o)) {
        void *p = PyLong_AsVoidPtr(o);
        if (!p && PyErr_Occurred()) ++*bad;
        return p;
    }
    PyObject *r = PyObject_CallMethodNoArgs(o, s_data_ptr);
    if (!r) {
        ++*bad;
        return NULL;
    }
    void *p = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    if (!p && PyErr_Occurred()) ++*bad;
    return p;
}

/* None (torch's current stream), a cudaStream_t as an int, or an object with cuda_stream. */
static wq_stream_t as_stream(PyObject *o, int *bad) {
    if (*bad) return NULL;
    if (PyLong_Check(o)) return (wq_stream_t)as_ptr(o, bad);
    PyObject *r = o == Py_None ? PyObject_CallNoArgs(current_stream)
                               : PyObject_GetAttr(o, s_cuda_stream);
    if (!r) {
        ++*bad;
        return NULL;
    }
    wq_stream_t s = (wq_stream_t)as_ptr(r, bad);
    Py_DECREF(r);
    return s;
}

/* None or a KvCache (its bytes are copied, so nothing is held). */
static const wq_kv_cache *as_cache(PyObject *o, wq_kv_cache *room, int *bad) {
    if (*bad || o == Py_None) return NULL;
    Py_buffer view;
    if (!PyObject_TypeCheck(o, (PyTypeObject *)cache_type)) {
        PyErr_Format(PyExc_TypeError, "cache: a KvCache is wanted, got %s", Py_TYPE(o)->tp_name);
        ++*bad;
        return NULL;
    }
    if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE) != 0) {
        ++*bad;
        return NULL;
    }
    if (view.len == (Py_ssize_t)sizeof(*room)) {
        *room = *(const wq_kv_cache *)view.buf;
    } else {
        PyErr_SetString(PyExc_TypeError, "cache: not the size of a wq_kv_cache");
        ++*bad;
    }
    PyBuffer_Release(&view);
    return room;
}

static int count_is(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return 1;
    PyErr_Format(PyExc_TypeError, "%zd arguments are wanted, got %zd", want, n);
    return 0;
}

#define I(k) as_int(a[k], &bad)
#define L(k) as_i64(a[k], &bad)
#define P(k) as_ptr(a[k], &bad)
#define CALL(expression)                  \
    if (bad) return NULL;                 \
    wq_status st;                         \
    Py_BEGIN_ALLOW_THREADS st = expression; \
    Py_END_ALLOW_THREADS return PyLong_FromLong(st)

static PyObject *rope(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    int bad = 0;
    if (!count_is(n, 13)) return NULL;
    const int rows = I(0), heads = I(1), dim = I(2), rot = I(3), table_rows = I(9);
    const unsigned flags = (unsigned)I(4);
    const float *x = P(5), *table = P(8);
    const int64_t x_stride = L(6), out_stride = L(11);
    const int32_t *pos = P(7);
    float *out = P(10);
    const wq_stream_t s = as_stream(a[12], &bad);
    CALL(f_rope(rows, heads, dim, rot, flags, x, x_stride, pos, table, table_rows, out, out_stride,
                s));
}

static PyObject *append(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    int bad = 0;
    if (!count_is(n, 25)) return NULL;
    wq_kv_cache room;
    const wq_kv_cache *cache = as_cache(a[0], &room, &bad);
    const int n_tok = I(1), h_q = I(2), rot = I(3), table_rows = I(13), n_seq = I(14);
    const unsigned flags = (unsigned)I(4);
    const float *q = P(5), *k = P(7), *v = P(9), *table = P(12);
    const int64_t q_stride = L(6), k_stride = L(8), v_stride = L(10);
    const int32_t *pos = P(11), *seq = P(15), *slot = P(16), *pages = P(17);
    const int max_pages = I(18);
    float *q_out = P(19), *acc = P(21);
    const int64_t q_out_stride = L(20), acc_stride = L(23);
    int32_t *slot_pos = P(22);
    const wq_stream_t s = as_stream(a[24], &bad);
    CALL(f_append(cache, n_tok, h_q, rot, flags, q, q_stride, k, k_stride, v, v_stride, pos, table,
                  table_rows, n_seq, seq, slot, pages, max_pages, q_out, q_out_stride, acc,
                  slot_pos, acc_stride, s));
}

static PyObject *attn(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    int bad = 0;
    if (!count_is(n, 21)) return NULL;
    wq_kv_cache cache_room;
    const wq_kv_cache *cache = as_cache(a[0], &cache_room, &bad);
    const int n_seq = I(1), h_q = I(2), window = I(4), max_pages = I(8);
    const float scale = as_float(a[3], &bad);
    const float *q = P(5), *mask = P(10), *acc_in = P(15);
    const int64_t q_stride = L(6), mask_stride = L(11), out_stride = L(13), acc_stride = L(17);
    const int32_t *pages = P(7), *lens = P(9);
    float *out = P(12), *lse = P(14), *acc_out = P(16);
    void *room = P(18);
    const size_t bytes = (size_t)L(19);
    const wq_stream_t s = as_stream(a[20], &bad);
    CALL(f_attn(cache, n_seq, h_q, scale, window, q, q_stride, pages, max_pages, lens, mask,
                mask_stride, out, out_stride, lse, acc_in, acc_out, acc_stride, room, bytes, s));
}

static PyObject *evict(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    int bad = 0;
    if (!count_is(n, 18)) return NULL;
    wq_kv_cache cache_room;
    const wq_kv_cache *cache = as_cache(a[0], &cache_room, &bad);
    const int n_seq = I(1), max_pages = I(3), keep = I(6), sinks = I(7), recent = I(8);
    const int32_t *pages = P(2), *lens = P(4), *seen = P(5), *slot_pos = P(10);
    const float *acc = P(9);
    float *acc_out = P(11);
    int32_t *pos_out = P(12), *lens_out = P(14);
    const int64_t acc_stride = L(13);
    void *room = P(15);
    const size_t bytes = (size_t)L(16);
    const wq_stream_t s = as_stream(a[17], &bad);
    CALL(f_evict(cache, n_seq, pages, max_pages, lens, seen, keep, sinks, recent, acc, slot_pos,
                 acc_out, pos_out, acc_stride, lens_out, room, bytes, s));
}

/* bind(rope, append, attn, evict, current_stream, KvCache): the first four are addresses. */
static PyObject *bind(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    int bad = 0;
    if (!count_is(n, 6)) return NULL;
    void *f[4];
    for (int i = 0; i < 4; ++i) f[i] = P(i);
    if (!bad && !PyType_Check(a[5])) {
        PyErr_SetString(PyExc_TypeError, "KvCache: a type is wanted");
        ++bad;
    }
    if (bad) return NULL;
    f_rope = (__typeof__(f_rope))f[0];
    f_append = (__typeof__(f_append))f[1];
    f_attn = (__typeof__(f_attn))f[2];
    f_evict = (__typeof__(f_evict))f[3];
    Py_INCREF(a[4]);
    Py_XSETREF(current_stream, a[4]);
    Py_INCREF(a[5]);
    Py_XSETREF(cache_type, a[5]);
    Py_RETURN_NONE;
}

#define FAST(name, f) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {FAST("bind", bind),
                                FAST("wq_rope", rope),
                                FAST("wq_kv_append", append),
                                FAST("wq_attn_paged", attn),
                                FAST("wq_kv_evict", evict),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_wq_calls", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__wq_calls(void) {
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    if (!s_data_ptr || !s_cuda_stream) return NULL;
    return PyModule_Create(&module);
}
