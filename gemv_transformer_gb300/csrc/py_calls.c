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
#include <string.h>

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
static wq_status (*f_norm)(int, int, int, const wq_head_norm *, const wq_rope_axes *, const float *,
                           int64_t, int, void *, int64_t, wq_stream_t);
static wq_status (*f_norm_grad)(int, int, int, const wq_head_norm *, const wq_rope_axes *,
                                const float *, int64_t, const float *, int64_t, float *, int64_t,
                                float *, float *, void *, size_t, wq_stream_t);
static wq_status (*f_append_norm)(const wq_kv_cache *, int, int, const wq_head_norm *,
                                  const wq_head_norm *, const wq_rope_axes *, const float *,
                                  int64_t, const float *, int64_t, const float *, int64_t, int,
                                  const int32_t *, const int32_t *, const int32_t *, int, int,
                                  void *, int64_t, float *, int32_t *, int64_t, wq_stream_t);
static wq_status (*f_tokens)(const wq_kv_cache *, int, int, int, float, const wq_attn_form *, int,
                             const void *, int64_t, const int32_t *, const int32_t *, int,
                             const int32_t *, int, void *, int64_t, float *, void *, size_t,
                             wq_stream_t);
static wq_status (*f_accept)(const wq_kv_cache *, int, int, int, const int32_t *, int,
                             const int32_t *, const int32_t *, const int32_t *, const int32_t *,
                             const int32_t *, int32_t *, int32_t *, int32_t *, int32_t *,
                             wq_stream_t);
static PyObject *current_stream; /* () -> int */
static PyObject *cache_type;     /* KvCache */
static PyObject *norm_type, *axes_type, *form_type; /* HeadNorm, RopeAxes, AttnForm */
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

/* None or a structure of `type` (its bytes are copied, so nothing is held). */
static void *as_struct(PyObject *o, PyObject *type, const char *what, void *room, size_t size,
                       int *bad) {
    if (*bad || o == Py_None) return NULL;
    Py_buffer view;
    if (!type || !PyObject_TypeCheck(o, (PyTypeObject *)type)) {
        PyErr_Format(PyExc_TypeError, "%s is wanted, got %s", what, Py_TYPE(o)->tp_name);
        ++*bad;
        return NULL;
    }
    if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE) != 0) {
        ++*bad;
        return NULL;
    }
    if (view.len == (Py_ssize_t)size) {
        memcpy(room, view.buf, size);
    } else {
        PyErr_Format(PyExc_TypeError, "%s: not the size of the C structure", what);
        ++*bad;
    }
    PyBuffer_Release(&view);
    return room;
}
static const wq_kv_cache *as_cache(PyObject *o, wq_kv_cache *room, int *bad) {
    return as_struct(o, cache_type, "cache: a KvCache", room, sizeof(*room), bad);
}
static const wq_head_norm *as_norm(PyObject *o, wq_head_norm *room, int *bad) {
    return as_struct(o, norm_type, "norm: a HeadNorm", room, sizeof(*room), bad);
}
static const wq_rope_axes *as_axes(PyObject *o, wq_rope_axes *room, int *bad) {
    return as_struct(o, axes_type, "rope: a RopeAxes", room, sizeof(*room), bad);
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

static PyObject *norm_rope(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    int bad = 0;
    if (!count_is(n, 11)) return NULL;
    wq_head_norm norm_room;
    wq_rope_axes axes_room;
    const int rows = I(0), heads = I(1), dim = I(2);
    const wq_head_norm *norm = as_norm(a[3], &norm_room, &bad);
    const wq_rope_axes *axes = as_axes(a[4], &axes_room, &bad);
    const float *x = P(5);
    const int64_t x_stride = L(6);
    const int type = I(7);
    void *out = P(8);
    const int64_t out_stride = L(9);
    const wq_stream_t s = as_stream(a[10], &bad);
    CALL(f_norm(rows, heads, dim, norm, axes, x, x_stride, type, out, out_stride, s));
}

static PyObject *norm_rope_grad(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    int bad = 0;
    if (!count_is(n, 16)) return NULL;
    wq_head_norm norm_room;
    wq_rope_axes axes_room;
    const int rows = I(0), heads = I(1), dim = I(2);
    const wq_head_norm *norm = as_norm(a[3], &norm_room, &bad);
    const wq_rope_axes *axes = as_axes(a[4], &axes_room, &bad);
    const float *x = P(5), *g = P(7);
    const int64_t x_stride = L(6), g_stride = L(8), gx_stride = L(10);
    float *gx = P(9), *gw = P(11), *gb = P(12);
    void *room = P(13);
    const size_t bytes = (size_t)L(14);
    const wq_stream_t s = as_stream(a[15], &bad);
    CALL(f_norm_grad(rows, heads, dim, norm, axes, x, x_stride, g, g_stride, gx, gx_stride, gw, gb,
                     room, bytes, s));
}

static PyObject *append_norm(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    int bad = 0;
    if (!count_is(n, 24)) return NULL;
    wq_kv_cache cache_room;
    wq_head_norm q_room, k_room;
    wq_rope_axes axes_room;
    const wq_kv_cache *cache = as_cache(a[0], &cache_room, &bad);
    const int n_tok = I(1), h_q = I(2), n_seq = I(12), max_pages = I(16), type = I(17);
    const wq_head_norm *q_norm = as_norm(a[3], &q_room, &bad);
    const wq_head_norm *k_norm = as_norm(a[4], &k_room, &bad);
    const wq_rope_axes *axes = as_axes(a[5], &axes_room, &bad);
    const float *q = P(6), *k = P(8), *v = P(10);
    const int64_t q_stride = L(7), k_stride = L(9), v_stride = L(11);
    const int32_t *seq = P(13), *slot = P(14), *pages = P(15);
    void *q_out = P(18);
    float *acc = P(20);
    const int64_t q_out_stride = L(19), acc_stride = L(22);
    int32_t *slot_pos = P(21);
    const wq_stream_t s = as_stream(a[23], &bad);
    CALL(f_append_norm(cache, n_tok, h_q, q_norm, k_norm, axes, q, q_stride, k, k_stride, v,
                       v_stride, n_seq, seq, slot, pages, max_pages, type, q_out, q_out_stride,
                       acc, slot_pos, acc_stride, s));
}

static PyObject *tokens(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    int bad = 0;
    if (!count_is(n, 20)) return NULL;
    wq_kv_cache cache_room;
    wq_attn_form form_room;
    const wq_kv_cache *cache = as_cache(a[0], &cache_room, &bad);
    const int n_seq = I(1), n_tok = I(2), h_q = I(3), q_type = I(6), max_pages = I(11);
    const float scale = as_float(a[4], &bad);
    const wq_attn_form *form =
        as_struct(a[5], form_type, "form: an AttnForm", &form_room, sizeof(form_room), &bad);
    const void *q = P(7);
    const int64_t q_stride = L(8), out_stride = L(15);
    const int32_t *starts = P(9), *pages = P(10), *lens = P(12);
    const int out_type = I(13);
    void *out = P(14), *room = P(17);
    float *lse = P(16);
    const size_t bytes = (size_t)L(18);
    const wq_stream_t s = as_stream(a[19], &bad);
    CALL(f_tokens(cache, n_seq, n_tok, h_q, scale, form, q_type, q, q_stride, starts, pages,
                  max_pages, lens, out_type, out, out_stride, lse, room, bytes, s));
}

/* The caches are an array of KvCache, held over the call; the count beside it is its length. */
static PyObject *accept_path(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    int bad = 0;
    if (!count_is(n, 16)) return NULL;
    const int count = I(1), n_seq = I(2), n_tok = I(3), max_pages = I(5);
    const int32_t *pages = P(4), *starts = P(6), *parent = P(7), *drafted = P(8), *choice = P(9);
    const int32_t *lens = P(10);
    int32_t *path = P(11), *accepted = P(12), *next = P(13), *lens_out = P(14);
    const wq_stream_t s = as_stream(a[15], &bad);
    if (bad) return NULL;
    PyObject *type = PyObject_GetAttrString(a[0], "_type_");
    const int known = type && type == cache_type;
    Py_XDECREF(type);
    if (!known) {
        PyErr_Format(PyExc_TypeError, "caches: an array of KvCache is wanted, got %s",
                     Py_TYPE(a[0])->tp_name);
        return NULL;
    }
    Py_buffer view;
    if (PyObject_GetBuffer(a[0], &view, PyBUF_SIMPLE) != 0) return NULL;
    if (count < 0 || view.len != (Py_ssize_t)sizeof(wq_kv_cache) * count) {
        PyBuffer_Release(&view);
        PyErr_SetString(PyExc_TypeError, "caches: not as many as their count");
        return NULL;
    }
    wq_status st;
    Py_BEGIN_ALLOW_THREADS st = f_accept(view.buf, count, n_seq, n_tok, pages, max_pages, starts,
                                         parent, drafted, choice, lens, path, accepted, next,
                                         lens_out, s);
    Py_END_ALLOW_THREADS PyBuffer_Release(&view);
    return PyLong_FromLong(st);
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

/* bind_tokens(norm_rope, norm_rope_grad, kv_append_norm, attn_tokens, kv_accept, HeadNorm, RopeAxes,
 * AttnForm): the first five are addresses. */
static PyObject *bind_tokens(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    int bad = 0;
    if (!count_is(n, 8)) return NULL;
    void *f[5];
    for (int i = 0; i < 5; ++i) f[i] = P(i);
    for (int i = 5; i < 8 && !bad; ++i)
        if (!PyType_Check(a[i])) {
            PyErr_SetString(PyExc_TypeError, "HeadNorm, RopeAxes, AttnForm: types are wanted");
            ++bad;
        }
    if (bad) return NULL;
    f_norm = (__typeof__(f_norm))f[0];
    f_norm_grad = (__typeof__(f_norm_grad))f[1];
    f_append_norm = (__typeof__(f_append_norm))f[2];
    f_tokens = (__typeof__(f_tokens))f[3];
    f_accept = (__typeof__(f_accept))f[4];
    Py_INCREF(a[5]);
    Py_XSETREF(norm_type, a[5]);
    Py_INCREF(a[6]);
    Py_XSETREF(axes_type, a[6]);
    Py_INCREF(a[7]);
    Py_XSETREF(form_type, a[7]);
    Py_RETURN_NONE;
}

#define FAST(name, f) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {FAST("bind", bind),
                                FAST("wq_rope", rope),
                                FAST("wq_kv_append", append),
                                FAST("wq_attn_paged", attn),
                                FAST("wq_kv_evict", evict),
                                FAST("bind_tokens", bind_tokens),
                                FAST("wq_norm_rope", norm_rope),
                                FAST("wq_norm_rope_grad", norm_rope_grad),
                                FAST("wq_kv_append_norm", append_norm),
                                FAST("wq_attn_tokens", tokens),
                                FAST("wq_kv_accept", accept_path),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_wq_calls", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__wq_calls(void) {
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    if (!s_data_ptr || !s_cuda_stream) return NULL;
    return PyModule_Create(&module);
}
