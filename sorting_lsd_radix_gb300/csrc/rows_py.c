/*
 * The row operators' calls from Python without ctypes: each function takes an
 * operator's tensors, tests them in the way of gbsort.py, and calls the C ABI.
 * A small call is bound by what the host does before its launch; here that is
 * about a microsecond (a tensor's address, shape, strides, type and device are
 * five calls of torch's own methods), and three in Python.
 *
 * A function returns the C call's status, or -1 where the arguments are not of
 * the plain kind (another type, layout or device, a work buffer that is too
 * small): gbsort.py then takes its own way, which says what is wrong or makes
 * what is missing.  Nothing is kept between calls.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "gbsort.h"

enum { T_F32, T_F16, T_BF16, T_I32, T_I64, T_TYPES };

static PyObject *g_types[T_TYPES], *g_raw_stream, *g_current_device, *g_bool, *g_uint8;
static PyObject *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_get_device, *s_numel, *s_is_contiguous, *s_element_size;

/* the C ABI's functions, by their addresses in the loaded library */
static gbs_status (*f_sort)(void *, size_t *, gbs_key_type, const void *, size_t, size_t, size_t, int64_t, size_t, size_t,
                            int32_t *, int32_t *, int32_t *, int32_t *, void *);
static gbs_status (*f_dispatch)(void *, size_t *, gbs_row_type, const void *, size_t, size_t, gbs_key_type, const void *,
                                size_t, size_t, size_t, int64_t, size_t, size_t, void *, size_t, int32_t *, int32_t *,
                                int32_t *, int32_t *, void *);
static gbs_status (*f_gather)(gbs_row_type, const void *, size_t, size_t, size_t, size_t, const int32_t *, const int32_t *,
                              size_t, void *, size_t, void *);
static gbs_status (*f_combine)(gbs_row_type, const void *, size_t, size_t, const int32_t *, gbs_row_type, const void *, size_t,
                               size_t, size_t, void *, size_t, void *);
static gbs_status (*f_combine_grad)(gbs_row_type, const void *, size_t, const void *, size_t, size_t, const int32_t *,
                                    const int32_t *, gbs_row_type, const void *, size_t, size_t, size_t, void *, size_t,
                                    void *, void *);
static gbs_status (*f_lookup)(gbs_row_type, const void *, size_t, size_t, gbs_key_type, const void *, size_t, int64_t, float,
                              size_t, void *, size_t, void *);
static gbs_status (*f_grad)(void *, size_t *, gbs_row_type, const void *, size_t, gbs_key_type, const void *, size_t, int64_t,
                            int64_t, float, size_t, size_t, gbs_row_type, void *, size_t, int, void *);

static gbs_status (*f_route)(gbs_row_type, const void *, size_t, size_t, size_t, size_t, gbs_score_type, const float *, size_t,
                             size_t, size_t, int, float, gbs_key_type, void *, gbs_row_type, void *, void *);
static gbs_status (*f_route_grad)(gbs_row_type, gbs_row_type, const void *, const void *, size_t, size_t, size_t, size_t,
                                  gbs_key_type, const void *, gbs_score_type, int, float, void *, size_t, void *);
static gbs_status (*f_select)(void *, size_t *, gbs_row_type, const void *, size_t, size_t, size_t, size_t, const float *,
                              const uint8_t *, int32_t, size_t, float *, int32_t *, int32_t *, void *);
static gbs_status (*f_reorder)(const void *, const size_t *, void *, const size_t *, size_t, size_t, size_t, size_t, size_t,
                               size_t, const int32_t *, void *);

/* A tensor of one or two dimensions. */
typedef struct {
    void *ptr;
    int type, dims;
    long dev;
    Py_ssize_t n[2], s[2];
} Tensor;

static int pair(PyObject *t, Py_ssize_t *out) {
    int i, dims;
    if (t == NULL || !PyTuple_Check(t)) {
        Py_XDECREF(t);
        return -1;
    }
    dims = (int)PyTuple_GET_SIZE(t);
    if (dims == 1 || dims == 2)
        for (i = 0; i < dims; ++i) out[i] = PyLong_AsSsize_t(PyTuple_GET_ITEM(t, i));
    else
        dims = -1;
    Py_DECREF(t);
    return dims;
}

/* One of T_*, or -1. */
static int type_of(PyObject *o) {
    PyObject *x = PyObject_GetAttr(o, s_dtype);
    int i;
    if (x == NULL) {
        PyErr_Clear();
        return -1;
    }
    for (i = 0; i < T_TYPES && x != g_types[i]; ++i) {}
    Py_DECREF(x);
    return i < T_TYPES ? i : -1;
}

/* 0, or -1 (with no exception set) for anything but a tensor of 1 or 2 dimensions and a known type. */
static int tensor(PyObject *o, Tensor *t) {
    PyObject *x;
    t->n[1] = t->s[1] = 1;
    if ((t->type = type_of(o)) < 0) return -1;
    if ((t->dims = pair(PyObject_GetAttr(o, s_shape), t->n)) < 0) goto fail;
    if (pair(PyObject_CallMethodNoArgs(o, s_stride), t->s) != t->dims) goto fail;
    if ((x = PyObject_CallMethodNoArgs(o, s_get_device)) == NULL) goto fail;
    t->dev = PyLong_AsLong(x);
    Py_DECREF(x);
    if ((x = PyObject_CallMethodNoArgs(o, s_data_ptr)) == NULL) goto fail;
    t->ptr = PyLong_AsVoidPtr(x);
    Py_DECREF(x);
    if (!PyErr_Occurred()) return 0;
fail:
    PyErr_Clear();
    return -1;
}

/* What a method without arguments says, as an integer; -1 (with no exception set) where it says nothing. */
static int64_t says(PyObject *o, PyObject *method) {
    PyObject *x = PyObject_CallMethodNoArgs(o, method);
    const int64_t v = x ? PyLong_AsLongLong(x) : -1;
    Py_XDECREF(x);
    if (v == -1) PyErr_Clear();
    return v;
}
static void *address(PyObject *o) {
    PyObject *x = PyObject_CallMethodNoArgs(o, s_data_ptr);
    void *p = x ? PyLong_AsVoidPtr(x) : NULL;
    Py_XDECREF(x);
    if (p == NULL) PyErr_Clear();
    return p;
}

/* Values that lie one after another, of any shape: of one of the types first .. last, `count` of them where that is not
   negative.  Their number, or -1. */
static int64_t values(PyObject *o, Tensor *t, long dev, int first, int last, int64_t count) {
    int64_t n;
    t->type = type_of(o);
    if (t->type < first || t->type > last || (n = says(o, s_numel)) < 0 || (count >= 0 && n != count)) return -1;
    if (says(o, s_get_device) != dev || says(o, s_is_contiguous) != 1) return -1;
    t->ptr = address(o);
    return n;
}

/* A work buffer's address on the device `dev` and its size, or NULL: also for a strided or expanded tensor, which has
   fewer bytes behind it than elements. */
static void *work_buffer(PyObject *o, long dev, size_t *bytes) {
    const int64_t n = says(o, s_numel);
    *bytes = n > 0 ? (size_t)n : 0;
    return says(o, s_get_device) == dev && says(o, s_is_contiguous) == 1 ? address(o) : NULL;
}

/* Rows with unit stride: the row type, or -1. */
static int matrix(PyObject *o, Tensor *t, long dev) {
    if (tensor(o, t) != 0 || t->dims != 2 || t->type > T_BF16) return -1;
    if ((t->n[1] > 1 && t->s[1] != 1) || t->s[0] < 0 || (dev >= 0 && t->dev != dev)) return -1;
    return t->type;
}

/* Neighbouring values of one of the types first .. last, `count` of them where that is not negative. */
static int plain(PyObject *o, Tensor *t, long dev, int first, int last, Py_ssize_t count) {
    if (tensor(o, t) != 0 || t->type < first || t->type > last || (dev >= 0 && t->dev != dev)) return -1;
    if (count >= 0 && t->n[0] * t->n[1] != count) return -1;
    if (t->n[0] * t->n[1] == 0) return 0;
    if (t->dims == 2 && ((t->n[1] > 1 && t->s[1] != 1) || (t->n[0] > 1 && t->s[0] != t->n[1]))) return -1;
    return t->dims == 1 && t->n[0] > 1 && t->s[0] != 1 ? -1 : 0;
}

static int integer(PyObject *o, int64_t *out) {
    *out = PyLong_AsLongLong(o);
    if (*out != -1 || !PyErr_Occurred()) return 0;
    PyErr_Clear();
    return -1;
}

/* The same for a value of 32 bits. */
static int integer32(PyObject *o, int64_t *out) { return integer(o, out) != 0 || *out < INT32_MIN || *out > INT32_MAX ? -1 : 0; }

static int number(PyObject *o, float *out) {
    const double x = PyFloat_AsDouble(o);
    *out = (float)x;
    if (x != -1.0 || !PyErr_Occurred()) return 0;
    PyErr_Clear();
    return -1;
}

/* The current stream of `dev`, which has to be the current device. */
static int stream_of(long dev, void **stream) {
    PyObject *x = PyObject_CallNoArgs(g_current_device), *n;
    long now = x ? PyLong_AsLong(x) : -1;
    Py_XDECREF(x);
    if (dev < 0 || now != dev) goto fail;
    if ((n = PyLong_FromLong(dev)) == NULL) goto fail;
    x = PyObject_CallOneArg(g_raw_stream, n);
    Py_DECREF(n);
    if (x == NULL) goto fail;
    *stream = PyLong_AsVoidPtr(x);
    Py_DECREF(x);
    if (!PyErr_Occurred()) return 0;
fail:
    PyErr_Clear();
    return -1;
}

static PyObject *done(gbs_status st) { return PyLong_FromLong(st == GBS_ERR_TEMP_TOO_SMALL ? -1 : (long)st); }
static PyObject *other(void) { return PyLong_FromLong(-1); }
static gbs_key_type id_type(const Tensor *t) { return t->type == T_I64 ? GBS_I64 : GBS_I32; }

/* (slot_of_row, row_of_slot, offsets, counts) of an order of ids[tokens, top_k]; num_rows: as slot_of_row has. */
static int order(PyObject *plan, const Tensor *ids, int64_t experts, int64_t *num_rows, Tensor *p) {
    if (ids->dims != 2 || !PyTuple_Check(plan) || PyTuple_GET_SIZE(plan) != 4 || experts < 1) return -1;
    if ((*num_rows = values(PyTuple_GET_ITEM(plan, 0), &p[0], ids->dev, T_I32, T_I32, -1)) < 0) return -1;
    if (values(PyTuple_GET_ITEM(plan, 1), &p[1], ids->dev, T_I32, T_I32, ids->n[0] * ids->n[1]) < 0) return -1;
    if (values(PyTuple_GET_ITEM(plan, 2), &p[2], ids->dev, T_I32, T_I32, experts + 1) < 0) return -1;
    return values(PyTuple_GET_ITEM(plan, 3), &p[3], ids->dev, T_I32, T_I32, experts) < 0 ? -1 : 0;
}

/* sort(ids, experts, first, align, plan, temp); dispatch(..., x, rows) */
static PyObject *sort_or_dispatch(PyObject *const *a, int rows_too) {
    Tensor ids, p[4], x, rows;
    int64_t experts, first, align, num_rows;
    size_t have;
    void *stream, *work;
    if (plain(a[0], &ids, -1, T_I32, T_I64, -1) != 0 || integer(a[1], &experts) || integer(a[2], &first) || integer(a[3], &align))
        return other();
    if (align < 1 || order(a[4], &ids, experts, &num_rows, p) != 0) return other();
    if ((work = work_buffer(a[5], ids.dev, &have)) == NULL) return other();
    if (rows_too) {
        if (matrix(a[6], &x, ids.dev) < 0 || matrix(a[7], &rows, ids.dev) != x.type) return other();
        if (x.n[0] != ids.n[0] || rows.n[0] != (Py_ssize_t)num_rows || rows.n[1] != x.n[1]) return other();
    }
    if (stream_of(ids.dev, &stream) != 0) return other();
    if (!rows_too)
        return done(f_sort(work, &have, id_type(&ids), ids.ptr, ids.n[0], ids.n[1], experts, first, align, num_rows, p[0].ptr,
                           p[1].ptr, p[2].ptr, p[3].ptr, stream));
    return done(f_dispatch(work, &have, (gbs_row_type)x.type, x.ptr, x.s[0], x.n[1], id_type(&ids), ids.ptr, ids.n[0], ids.n[1],
                           experts, first, align, num_rows, rows.ptr, rows.s[0], p[0].ptr, p[1].ptr, p[2].ptr, p[3].ptr, stream));
}
static PyObject *py_sort(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    return n == 6 ? sort_or_dispatch(a, 0) : other();
}
static PyObject *py_dispatch(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    return n == 8 ? sort_or_dispatch(a, 1) : other();
}

/* gather(x, slot_of_row, row_of_slot, rows) */
static PyObject *py_gather(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Tensor x, slot_of, row_of, rows;
    void *stream;
    (void)self;
    if (n != 4 || matrix(a[0], &x, -1) < 0 || plain(a[2], &row_of, x.dev, T_I32, T_I32, -1) != 0 || row_of.dims != 2) return other();
    if (matrix(a[3], &rows, x.dev) != x.type || rows.n[1] != x.n[1] || row_of.n[0] != x.n[0]) return other();
    if (values(a[1], &slot_of, x.dev, T_I32, T_I32, rows.n[0]) < 0 || stream_of(x.dev, &stream) != 0) return other();
    return done(f_gather((gbs_row_type)x.type, x.ptr, x.s[0], x.n[0], row_of.n[1], x.n[1], slot_of.ptr, row_of.ptr, rows.n[0],
                         rows.ptr, rows.s[0], stream));
}

/* combine(rows, row_of_slot, weights or None, out) */
static PyObject *py_combine(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Tensor rows, row_of, w, out;
    void *stream;
    (void)self;
    if (n != 4 || matrix(a[0], &rows, -1) < 0 || plain(a[1], &row_of, rows.dev, T_I32, T_I32, -1) != 0 || row_of.dims != 2) return other();
    w.ptr = NULL;
    w.type = T_F32;
    if (a[2] != Py_None && (values(a[2], &w, rows.dev, T_F32, T_BF16, row_of.n[0] * row_of.n[1]) < 0 ||
                            (w.type != T_F32 && w.type != rows.type)))
        return other();
    if (matrix(a[3], &out, rows.dev) != rows.type || out.n[0] != row_of.n[0] || out.n[1] != rows.n[1]) return other();
    if (stream_of(rows.dev, &stream) != 0) return other();
    return done(f_combine((gbs_row_type)rows.type, rows.ptr, rows.s[0], rows.n[0], row_of.ptr, (gbs_row_type)w.type, w.ptr,
                          row_of.n[0], row_of.n[1], rows.n[1], out.ptr, out.s[0], stream));
}

/* combine_grad(d_out, rows, slot_of_row, row_of_slot, weights, d_rows, d_weights) */
static PyObject *py_combine_grad(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Tensor d_out, rows, slot_of, row_of, w, d_rows, d_w;
    void *stream;
    (void)self;
    if (n != 7 || matrix(a[1], &rows, -1) < 0 || plain(a[3], &row_of, rows.dev, T_I32, T_I32, -1) != 0 || row_of.dims != 2) return other();
    if (matrix(a[0], &d_out, rows.dev) != rows.type || d_out.n[0] != row_of.n[0] || d_out.n[1] != rows.n[1]) return other();
    if (matrix(a[5], &d_rows, rows.dev) != rows.type || d_rows.n[0] != rows.n[0] || d_rows.n[1] != rows.n[1]) return other();
    if (values(a[2], &slot_of, rows.dev, T_I32, T_I32, rows.n[0]) < 0) return other();
    if (values(a[4], &w, rows.dev, T_F32, T_BF16, row_of.n[0] * row_of.n[1]) < 0 || (w.type != T_F32 && w.type != rows.type)) return other();
    if (values(a[6], &d_w, rows.dev, w.type, w.type, row_of.n[0] * row_of.n[1]) < 0 || stream_of(rows.dev, &stream) != 0) return other();
    return done(f_combine_grad((gbs_row_type)rows.type, d_out.ptr, d_out.s[0], rows.ptr, rows.s[0], rows.n[0], slot_of.ptr, row_of.ptr,
                               (gbs_row_type)w.type, w.ptr, row_of.n[0], row_of.n[1], rows.n[1], d_rows.ptr, d_rows.s[0], d_w.ptr,
                               stream));
}

/* lookup(table, ids, scale, first_id, out) */
static PyObject *py_lookup(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Tensor table, ids, out;
    int64_t first;
    float scale;
    void *stream;
    (void)self;
    if (n != 5 || matrix(a[0], &table, -1) < 0 || plain(a[1], &ids, table.dev, T_I32, T_I64, -1) != 0 || ids.dims != 1) return other();
    if (number(a[2], &scale) || integer(a[3], &first)) return other();
    if (matrix(a[4], &out, table.dev) != table.type || out.n[0] != ids.n[0] || out.n[1] != table.n[1]) return other();
    if (stream_of(table.dev, &stream) != 0) return other();
    return done(f_lookup((gbs_row_type)table.type, table.ptr, table.s[0], table.n[0], id_type(&ids), ids.ptr, ids.n[0], first, scale,
                         table.n[1], out.ptr, out.s[0], stream));
}

/* grad(d_out, ids, grad, scale, first_id, padding_id, accumulate, temp) */
static PyObject *py_grad(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Tensor d_out, ids, grad;
    int64_t first, padding, add;
    float scale;
    void *stream, *temp;
    size_t have;
    (void)self;
    if (n != 8 || matrix(a[2], &grad, -1) < 0 || plain(a[1], &ids, grad.dev, T_I32, T_I64, -1) != 0 || ids.dims != 1) return other();
    if (matrix(a[0], &d_out, grad.dev) < 0 || d_out.n[0] != ids.n[0] || d_out.n[1] != grad.n[1]) return other();
    if (grad.type != T_F32 && grad.type != d_out.type) return other();
    if (number(a[3], &scale) || integer(a[4], &first) || integer(a[5], &padding) || integer(a[6], &add)) return other();
    if ((temp = work_buffer(a[7], grad.dev, &have)) == NULL || stream_of(grad.dev, &stream) != 0) return other();
    return done(f_grad(temp, &have, (gbs_row_type)d_out.type, d_out.ptr, d_out.s[0], id_type(&ids), ids.ptr, ids.n[0], first, padding,
                       scale, grad.n[0], grad.n[1], (gbs_row_type)grad.type, grad.ptr, grad.s[0], add != 0, stream));
}

/* route(logits, top_k, score_type, bias or None, num_groups, top_groups, group_top, renormalise, scale, ids, weights) */
static PyObject *py_route(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Tensor logits, bias, ids, w;
    int64_t top_k, score, groups, top_groups, group_top, renorm;
    float scale;
    void *stream;
    (void)self;
    if (n != 11 || matrix(a[0], &logits, -1) < 0 || integer(a[1], &top_k) || integer32(a[2], &score) || integer(a[4], &groups)) return other();
    if (integer(a[5], &top_groups) || integer(a[6], &group_top) || integer(a[7], &renorm) || number(a[8], &scale)) return other();
    if (top_k < 1 || groups < 1 || top_groups < 1 || group_top < 1) return other();
    bias.ptr = NULL;
    if (a[3] != Py_None && values(a[3], &bias, logits.dev, T_F32, T_F32, logits.n[1]) < 0) return other();
    if (plain(a[9], &ids, logits.dev, T_I32, T_I64, -1) != 0 || ids.dims != 2 || ids.n[0] != logits.n[0] || ids.n[1] != top_k) return other();
    if (plain(a[10], &w, logits.dev, T_F32, T_BF16, -1) != 0 || w.dims != 2 || w.n[0] != logits.n[0] || w.n[1] != top_k) return other();
    if ((w.type != T_F32 && w.type != logits.type) || stream_of(logits.dev, &stream) != 0) return other();
    return done(f_route((gbs_row_type)logits.type, logits.ptr, logits.s[0], logits.n[0], logits.n[1], top_k, (gbs_score_type)score,
                        (const float *)bias.ptr, groups, top_groups, group_top, renorm != 0, scale, id_type(&ids), ids.ptr,
                        (gbs_row_type)w.type, w.ptr, stream));
}

/* route_grad(d_weights, logits, ids, score_type, renormalise, scale, d_logits) */
static PyObject *py_route_grad(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Tensor d_w, logits, ids, d;
    int64_t score, renorm;
    float scale;
    void *stream;
    (void)self;
    if (n != 7 || matrix(a[1], &logits, -1) < 0 || integer32(a[3], &score) || integer(a[4], &renorm) || number(a[5], &scale)) return other();
    if (plain(a[2], &ids, logits.dev, T_I32, T_I64, -1) != 0 || ids.dims != 2 || ids.n[0] != logits.n[0] || ids.n[1] < 1) return other();
    if (plain(a[0], &d_w, logits.dev, T_F32, T_BF16, -1) != 0 || d_w.dims != 2 || d_w.n[0] != ids.n[0] || d_w.n[1] != ids.n[1]) return other();
    if (d_w.type != T_F32 && d_w.type != logits.type) return other();
    if (matrix(a[6], &d, logits.dev) != logits.type || d.n[0] != logits.n[0] || d.n[1] != logits.n[1]) return other();
    if (stream_of(logits.dev, &stream) != 0) return other();
    return done(f_route_grad((gbs_row_type)logits.type, (gbs_row_type)d_w.type, d_w.ptr, logits.ptr, logits.s[0], logits.n[0], logits.n[1],
                             ids.n[1], id_type(&ids), ids.ptr, (gbs_score_type)score, renorm != 0, scale, d.ptr, d.s[0], stream));
}

/* beam_select(logits, scores, num_out, finished or None, end_id, (scores, beams, tokens), temp) */
static PyObject *py_beam_select(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Tensor logits, scores, out[3];
    int64_t count, end;
    size_t have;
    void *stream, *temp, *finished = NULL;
    int i;
    (void)self;
    if (n != 7 || matrix(a[0], &logits, -1) < 0 || plain(a[1], &scores, logits.dev, T_F32, T_F32, -1) != 0 || scores.dims != 2) return other();
    if (logits.n[0] != scores.n[0] * scores.n[1] || integer(a[2], &count) || integer32(a[4], &end)) return other();
    if (count < 1 || !PyTuple_Check(a[5]) || PyTuple_GET_SIZE(a[5]) != 3) return other();
    for (i = 0; i < 3; ++i)
        if (values(PyTuple_GET_ITEM(a[5], i), &out[i], logits.dev, i == 0 ? T_F32 : T_I32, i == 0 ? T_F32 : T_I32, scores.n[0] * count) < 0) return other();
    if (a[3] != Py_None) {
        PyObject *type = PyObject_GetAttr(a[3], s_dtype);
        if (type == NULL) PyErr_Clear();
        Py_XDECREF(type);
        if (type == NULL || (type != g_bool && type != g_uint8) || says(a[3], s_numel) != scores.n[0] * scores.n[1] ||
            says(a[3], s_get_device) != logits.dev || says(a[3], s_is_contiguous) != 1)
            return other();
        finished = address(a[3]);
        if (finished == NULL && scores.n[0] * scores.n[1] != 0) return other();
    }
    if ((temp = work_buffer(a[6], logits.dev, &have)) == NULL || stream_of(logits.dev, &stream) != 0) return other();
    return done(f_select(temp, &have, (gbs_row_type)logits.type, logits.ptr, logits.s[0], scores.n[0], scores.n[1], logits.n[1],
                         (const float *)scores.ptr, (const uint8_t *)finished, (int32_t)end, count, (float *)out[0].ptr,
                         (int32_t *)out[1].ptr, (int32_t *)out[2].ptr, stream));
}

enum { MOST_DIMS = 12 };

/* A tensor of any type and up to MOST_DIMS dimensions: their number, or -1. */
static int shape_of(PyObject *o, int64_t *size, int64_t *stride) {
    PyObject *n = PyObject_GetAttr(o, s_shape), *s = n ? PyObject_CallMethodNoArgs(o, s_stride) : NULL;
    int i, dims = -1;
    if (n && s && PyTuple_Check(n) && PyTuple_Check(s) && PyTuple_GET_SIZE(n) == PyTuple_GET_SIZE(s) && PyTuple_GET_SIZE(n) <= MOST_DIMS) {
        dims = (int)PyTuple_GET_SIZE(n);
        for (i = 0; i < dims; ++i) {
            size[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(n, i));
            stride[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(s, i));
        }
    }
    Py_XDECREF(n);
    Py_XDECREF(s);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return -1;
    }
    return dims;
}

/* Dimensions first .. last - 1 merged into as few as they can be in both tensors, the last first; their number. */
static int merged(const int64_t *size, const int64_t *s, const int64_t *t, int first, int last, int64_t (*dim)[3]) {
    int i, count = 0;
    for (i = last - 1; i >= first; --i) {
        if (size[i] == 1) continue;
        if (count > 0 && s[i] == dim[count - 1][1] * dim[count - 1][0] && t[i] == dim[count - 1][2] * dim[count - 1][0]) {
            dim[count - 1][0] *= size[i];
            continue;
        }
        dim[count][0] = size[i];
        dim[count][1] = s[i];
        dim[count++][2] = t[i];
    }
    return count;
}

/* beam_reorder(state, parents, dim, out: state for in place) */
static PyObject *py_beam_reorder(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Tensor parents;
    int64_t size[MOST_DIMS], s[MOST_DIMS], into[MOST_DIMS], t[MOST_DIMS], outer[MOST_DIMS][3], inner[MOST_DIMS][3], dim, bytes, length = 1, all = 1;
    int64_t many[3] = {1, 0, 0}, segment[3] = {1, 0, 0};
    size_t in[4], out[4];
    int dims, i, outers, inners;
    const long dev = n == 4 ? (long)says(a[0], s_get_device) : -1;
    void *stream, *from, *to;
    (void)self;
    if (n != 4 || dev < 0 || integer(a[2], &dim) || (dims = shape_of(a[0], size, s)) < 0 || dim < 0 || dim + 1 >= dims) return other();
    if (plain(a[1], &parents, dev, T_I32, T_I32, -1) != 0 || parents.dims != 2 || parents.n[0] != size[dim]) return other();
    if (a[3] == a[0]) {
        for (i = 0; i < dims; ++i) into[i] = size[i], t[i] = s[i];
    } else {
        PyObject *x = PyObject_GetAttr(a[0], s_dtype), *y = PyObject_GetAttr(a[3], s_dtype);
        const int same = x != NULL && x == y;
        Py_XDECREF(x);
        Py_XDECREF(y);
        PyErr_Clear();
        if (!same || shape_of(a[3], into, t) != dims || says(a[3], s_get_device) != dev) return other();
    }
    for (i = 0; i < dims; ++i) {
        all *= size[i];
        if (s[i] < 0 || t[i] < 0 || into[i] != (i == dim + 1 ? parents.n[1] : size[i])) return other();
    }
    outers = merged(size, s, t, 0, (int)dim, outer);
    inners = merged(size, s, t, (int)dim + 2, dims, inner);
    i = 0;
    if (inners > 0 && inner[0][1] == 1 && inner[0][2] == 1) length = inner[i++][0];
    if (outers > 1 || inners - i > 1 || (bytes = says(a[0], s_element_size)) < 1) return other();
    if (outers == 1) many[0] = outer[0][0], many[1] = outer[0][1], many[2] = outer[0][2];
    if (inners - i == 1) segment[0] = inner[i][0], segment[1] = inner[i][1], segment[2] = inner[i][2];
    in[0] = many[1] * bytes, in[1] = s[dim] * bytes, in[2] = s[dim + 1] * bytes, in[3] = segment[1] * bytes;
    out[0] = many[2] * bytes, out[1] = t[dim] * bytes, out[2] = t[dim + 1] * bytes, out[3] = segment[2] * bytes;
    from = address(a[0]);
    to = a[3] == a[0] ? from : address(a[3]);
    if (all == 0 || from == NULL || to == NULL || stream_of(dev, &stream) != 0) return other();
    return done(f_reorder(from, in, to, out, many[0], size[dim], size[dim + 1], parents.n[1], segment[0], length * bytes,
                          (const int32_t *)parents.ptr, stream));
}

/* setup_select(bool, uint8, addresses): what the operators that select need beside setup's */
static PyObject *py_setup_select(PyObject *self, PyObject *args) {
    PyObject *flag, *byte, *at;
    void **f[4] = {(void **)&f_route, (void **)&f_route_grad, (void **)&f_select, (void **)&f_reorder};
    int i;
    (void)self;
    if (!PyArg_ParseTuple(args, "OOO!", &flag, &byte, &PyTuple_Type, &at)) return NULL;
    if (PyTuple_GET_SIZE(at) != 4) {
        PyErr_SetString(PyExc_ValueError, "setup_select: four addresses");
        return NULL;
    }
    for (i = 0; i < 4; ++i)
        if ((*f[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(at, i))) == NULL)
            return PyErr_Occurred() ? NULL : PyErr_Format(PyExc_ValueError, "setup_select: a null address");
    Py_XSETREF(g_bool, Py_NewRef(flag));
    Py_XSETREF(g_uint8, Py_NewRef(byte));
    Py_RETURN_NONE;
}

/* setup(types, raw_stream, current_device, addresses): torch's types and functions, the C ABI's addresses */
static PyObject *py_setup(PyObject *self, PyObject *args) {
    PyObject *types, *raw, *dev, *at;
    void **f[7];
    int i;
    (void)self;
    if (!PyArg_ParseTuple(args, "O!OOO!", &PyTuple_Type, &types, &raw, &dev, &PyTuple_Type, &at)) return NULL;
    if (PyTuple_GET_SIZE(types) != T_TYPES || PyTuple_GET_SIZE(at) != 7) {
        PyErr_SetString(PyExc_ValueError, "setup: five types and seven addresses");
        return NULL;
    }
    f[0] = (void **)&f_sort;
    f[1] = (void **)&f_dispatch;
    f[2] = (void **)&f_gather;
    f[3] = (void **)&f_combine;
    f[4] = (void **)&f_combine_grad;
    f[5] = (void **)&f_lookup;
    f[6] = (void **)&f_grad;
    for (i = 0; i < 7; ++i)
        if ((*f[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(at, i))) == NULL) return PyErr_Occurred() ? NULL : PyErr_Format(PyExc_ValueError, "setup: a null address");
    for (i = 0; i < T_TYPES; ++i) Py_XSETREF(g_types[i], Py_NewRef(PyTuple_GET_ITEM(types, i)));
    Py_XSETREF(g_raw_stream, Py_NewRef(raw));
    Py_XSETREF(g_current_device, Py_NewRef(dev));
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"setup", py_setup, METH_VARARGS, NULL},
                                {"sort", (PyCFunction)(void (*)(void))py_sort, METH_FASTCALL, NULL},
                                {"dispatch", (PyCFunction)(void (*)(void))py_dispatch, METH_FASTCALL, NULL},
                                {"gather", (PyCFunction)(void (*)(void))py_gather, METH_FASTCALL, NULL},
                                {"combine", (PyCFunction)(void (*)(void))py_combine, METH_FASTCALL, NULL},
                                {"combine_grad", (PyCFunction)(void (*)(void))py_combine_grad, METH_FASTCALL, NULL},
                                {"lookup", (PyCFunction)(void (*)(void))py_lookup, METH_FASTCALL, NULL},
                                {"grad", (PyCFunction)(void (*)(void))py_grad, METH_FASTCALL, NULL},
                                {"setup_select", py_setup_select, METH_VARARGS, NULL},
                                {"route", (PyCFunction)(void (*)(void))py_route, METH_FASTCALL, NULL},
                                {"route_grad", (PyCFunction)(void (*)(void))py_route_grad, METH_FASTCALL, NULL},
                                {"beam_select", (PyCFunction)(void (*)(void))py_beam_select, METH_FASTCALL, NULL},
                                {"beam_reorder", (PyCFunction)(void (*)(void))py_beam_reorder, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rows", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__rows(void) {
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_numel = PyUnicode_InternFromString("numel");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_element_size = PyUnicode_InternFromString("element_size");
    if (!s_dtype || !s_shape || !s_stride || !s_data_ptr || !s_get_device || !s_numel || !s_is_contiguous || !s_element_size) return NULL;
    return PyModule_Create(&module);
}
