/* Marshalling of the decode calls (few-row products, routing, the MoE layer) and of the feed-forward
 * training calls (gated block, quantiser, Newton-Schulz) from torch tensors to the C ABI, for
 * binding.py.  Such a call takes a few microseconds on the device, and its
 * arguments cost as much through ctypes and Python attribute lookups (1 x 256 routing: 6.1 us a
 * call, of which the launch is 1.9).  Only Python's C API is used: tensors are asked through
 * their own methods.  A failed check raises AssertionError; the calls return the dg_status. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "dg.h"

typedef dg_status (*GemvFn)(const void *, int64_t, const void *, int64_t, const void *, const void *, int64_t, void *,
                            int64_t, int, int, int, void *, int64_t, int32_t *, void *);
typedef dg_status (*RouteFn)(const void *, int64_t, int, const float *, int32_t *, float *, int, int, int, int, int,
                             float, void *);
typedef dg_status (*LayerFn)(const void *, int64_t, const int32_t *, const float *, const void *, const void *,
                             const void *, const void *, const void *, int64_t, void *, int64_t, int, int, int, int,
                             int, void *, int64_t, int32_t *, void *);
typedef int64_t (*GemvBytesFn)(int, int, int);
typedef int64_t (*LayerBytesFn)(int, int, int, int, int);
typedef dg_status (*GatedFn)(const void *, int64_t, const void *, const void *, int64_t, const void *, void *, int64_t,
                             void *, int64_t, void *, int64_t, void *, int, int, int, int32_t *, void *);
typedef dg_status (*GatedGroupedFn)(const void *, int64_t, const void *, const void *, int64_t, const void *, void *,
                                    int64_t, void *, int64_t, void *, int64_t, void *, const int32_t *, int, int, int,
                                    int, int32_t *, void *);
typedef dg_status (*BackwardFn)(const void *, int64_t, const void *, const void *, int64_t, const void *, const void *,
                                int64_t, void *, int64_t, void *, int64_t, int, int, int, int32_t *, void *);
typedef dg_status (*BackwardGroupedFn)(const void *, int64_t, const void *, const void *, int64_t, const void *,
                                       const void *, int64_t, void *, int64_t, void *, int64_t, const int32_t *, int,
                                       int, int, int, int32_t *, void *);
typedef dg_status (*QuantizeFn)(const void *, int, int64_t, void *, int64_t, void *, void *, int64_t, void *, int, int,
                                const int *, int, void *);
typedef dg_status (*BlocksFn)(const void *, int, int64_t, int64_t, void *, int64_t, int64_t, void *, void *, int, int,
                              int, void *);
typedef dg_status (*SchulzFn)(const void *, int, int64_t, int64_t, void *, int64_t, int64_t, int, int, int, int, float,
                              float, float, float, void *, int64_t, int32_t *, void *);
typedef int64_t (*SchulzBytesFn)(int, int, int);
typedef int64_t (*PackedRowsFn)(const int *, int);

enum { GEMV_FP4, GEMV_FP8, GEMV_FP4_F32, GEMV_FP8_F32, ROUTE, LAYER_FP4, LAYER_FP8, GEMV_BYTES, LAYER_BYTES,
       GATED, GATED_GROUPED, BACKWARD, BACKWARD_GROUPED, QUANTIZE, BLOCKS, SCHULZ, SCHULZ_BYTES, PACKED_ROWS, FNS };
enum { BF16, F32, FP8, U8, I32, DTYPES };

static void *fns[FNS];
static PyObject *dtypes[DTYPES], *raw_stream, *current_device, *make_workspace;
static PyObject *s_data_ptr, *s_stride, *s_shape, *s_dtype, *s_is_contiguous, *s_get_device, *s_nbytes, *s_cuda_stream;

#define CHECK(cond)                                                       \
    do {                                                                  \
        if (!(cond)) {                                                    \
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_AssertionError, #cond); \
            goto fail;                                                    \
        }                                                                 \
    } while (0)

/* Shape (and strides) of a tensor of `dims` dimensions; 0 if it has others. */
typedef struct {
    int64_t n[3], stride[3];
    void *p;
} Tensor;

static int dims_of(PyObject *tuple, int dims, int64_t *out) {
    int i, ok = tuple && PyTuple_Check(tuple) && PyTuple_GET_SIZE(tuple) == dims;
    for (i = 0; ok && i < dims; ++i) {
        out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
        ok = out[i] >= 0 || !PyErr_Occurred();
    }
    Py_XDECREF(tuple);
    return ok;
}

static int pointer_of(PyObject *t, void **out) {
    PyObject *r = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!r) return 0;
    *out = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    return *out || !PyErr_Occurred();
}

static int is_dtype(PyObject *t, PyObject *dtype) {
    PyObject *r = PyObject_GetAttr(t, s_dtype);
    Py_XDECREF(r);   /* (the dtypes are held here) */
    return r == dtype;
}

static int is_contiguous(PyObject *t) {
    PyObject *r = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    Py_XDECREF(r);
    return r == Py_True;
}

static int shape_of(PyObject *t, int dims, Tensor *out) {
    return dims_of(PyObject_GetAttr(t, s_shape), dims, out->n) && pointer_of(t, &out->p);
}

static int strided(PyObject *t, int dims, Tensor *out) {
    return shape_of(t, dims, out) && dims_of(PyObject_CallMethodNoArgs(t, s_stride), dims, out->stride);
}

/* Elements of a contiguous tensor, from its bytes. */
static int64_t bytes_of(PyObject *t) {
    PyObject *r = PyObject_GetAttr(t, s_nbytes);
    const int64_t n = r ? PyLong_AsLongLong(r) : -1;
    Py_XDECREF(r);
    return n;
}

/* The status word, or NULL: the kernels OR into 4 bytes. */
static int status_of(PyObject *t, void **out) {
    *out = NULL;
    return t == Py_None || (is_dtype(t, dtypes[I32]) && is_contiguous(t) && bytes_of(t) >= 4 && pointer_of(t, out));
}

/* Row stride in elements; a single row's own length, for its stride says nothing (and need not
 * be one that rows may have). */
static int64_t row_stride(const Tensor *t) { return t->n[0] > 1 ? t->stride[0] : t->n[1]; }

/* Whether all tensors (NULL or None: not given) are on the current CUDA device, the one that the
 * library launches on: its kernels would fault on the pointer of any other. */
static int placed(PyObject *const *tensors, int n) {
    PyObject *d = PyObject_CallNoArgs(current_device), *r;
    long device, at;
    int i;
    if (!d) return 0;
    device = PyLong_AsLong(d);
    Py_DECREF(d);
    if (device == -1 && PyErr_Occurred()) return 0;
    for (i = 0; i < n; ++i) {
        if (!tensors[i] || tensors[i] == Py_None) continue;
        r = PyObject_CallMethodNoArgs(tensors[i], s_get_device);   /* (-1 on the host) */
        if (!r) return 0;
        at = PyLong_AsLong(r);
        Py_DECREF(r);
        if (at != device) {
            if (!PyErr_Occurred())
                PyErr_Format(PyExc_AssertionError, "operand on device %ld (-1: host), current device %ld", at, device);
            return 0;
        }
    }
    return 1;
}

static int stream_of(PyObject *stream, PyObject *on, void **out) {
    PyObject *d, *r;
    if (stream != Py_None) {
        r = PyObject_GetAttr(stream, s_cuda_stream);
    } else {
        d = PyObject_CallMethodNoArgs(on, s_get_device);
        r = d ? PyObject_CallOneArg(raw_stream, d) : NULL;
        Py_XDECREF(d);
    }
    if (!r) return 0;
    *out = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    return *out || !PyErr_Occurred();
}

/* The stream and the workspace of a call on `tensors`, which all have to be on the current device:
 * the caller's workspace, or one of `need` bytes (a new reference in *hold).  Where the library does
 * not take the sizes (`need` negative) or the workspace is too small, it refuses the call before
 * any device access: then no tensor's place counts, and no workspace is made. */
static int device_side(PyObject *const *tensors, int count, PyObject *given, int64_t need, PyObject *on, PyObject *stream,
                       PyObject **hold, void **p, int64_t *bytes, void **stream_out) {
    *p = *stream_out = NULL;
    *bytes = 0;
    if (given != Py_None) {
        if (!is_contiguous(given)) return 0;   /* its bytes would not be one range */
        *bytes = bytes_of(given);
        if (*bytes < 0 || !pointer_of(given, p)) return 0;
    }
    if (need < 0 || (given != Py_None && *bytes < need)) return 1;
    if (!placed(tensors, count) || !placed(&given, 1) || !stream_of(stream, on, stream_out)) return 0;
    if (given == Py_None) {
        PyObject *n, *args[3];
        if (need == 0) return 1;
        n = PyLong_FromLongLong(need);
        if (!n) return 0;
        args[0] = n;
        args[1] = on;
        args[2] = stream;
        given = *hold = PyObject_Vectorcall(make_workspace, args, 3, NULL);
        Py_DECREF(n);
        if (!given) return 0;
        *bytes = bytes_of(given);
        return *bytes >= 0 && pointer_of(given, p);
    }
    return 1;
}

static PyObject *gemv(PyObject *self, PyObject *const *arg, Py_ssize_t nargs) {
    Tensor a, b, d, c = {{0, 0, 0}, {0, 0, 0}, NULL};
    PyObject *hold = NULL, *dtype;
    void *sf, *ws, *status, *stream;
    int64_t m, n, k, ws_bytes;
    int which, fp4;
    dg_status st;
    CHECK(nargs == 9);
    which = (int)PyLong_AsLong(arg[0]);
    CHECK(which >= GEMV_FP4 && which <= GEMV_FP8_F32);
    fp4 = which == GEMV_FP4 || which == GEMV_FP4_F32;
    dtype = dtypes[which >= GEMV_FP4_F32 ? F32 : BF16];
    {
        PyObject *const ta = arg[1], *const tb = arg[2], *const sfb = arg[3], *const td = arg[4], *const tc = arg[5];
        CHECK(strided(ta, 2, &a) && strided(tb, 2, &b) && strided(td, 2, &d));
        m = a.n[0];
        k = a.n[1];
        n = b.n[0];
        CHECK(is_dtype(ta, dtypes[BF16]) && is_dtype(td, dtype) && is_dtype(sfb, dtypes[I32]));
        CHECK(is_dtype(tb, dtypes[fp4 ? U8 : FP8]) && (fp4 ? 2 : 1) * b.n[1] == k);
        CHECK(d.n[0] == m && d.n[1] == n && (d.stride[1] == 1 || n <= 1));
        CHECK((a.stride[1] == 1 && b.stride[1] == 1) || k <= 1);
        CHECK(m <= INT32_MAX && n <= INT32_MAX && k <= INT32_MAX);
        CHECK(is_contiguous(sfb) && bytes_of(sfb) >= (fp4 ? (k + 127) / 128 : (k + 511) / 512) * ((n + 3) / 4 * 4) * 4);
        CHECK(tc == Py_None ||
              (is_dtype(tc, dtype) && strided(tc, 2, &c) && c.n[0] == m && c.n[1] == n && (c.stride[1] == 1 || n <= 1)));
        CHECK(pointer_of(sfb, &sf) && status_of(arg[7], &status));
        PyObject *const on_device[] = {ta, tb, sfb, td, tc, arg[7]};
        CHECK(device_side(on_device, 6, arg[6], ((GemvBytesFn)fns[GEMV_BYTES])((int)m, (int)n, (int)k), td, arg[8], &hold,
                          &ws, &ws_bytes, &stream));
    }
    Py_BEGIN_ALLOW_THREADS
    st = ((GemvFn)fns[which])(a.p, row_stride(&a), b.p, row_stride(&b), sf, c.p, c.p ? row_stride(&c) : 0, d.p,
                              row_stride(&d), (int)m, (int)n, (int)k, ws, ws_bytes, (int32_t *)status, stream);
    Py_END_ALLOW_THREADS
    Py_XDECREF(hold);
    return PyLong_FromLong(st);
fail:
    Py_XDECREF(hold);
    return NULL;
}

static PyObject *route(PyObject *self, PyObject *const *arg, Py_ssize_t nargs) {
    Tensor logits, ids, weights, bias = {{0, 0, 0}, {0, 0, 0}, NULL};
    void *stream;
    double scale;
    int f32, sigmoid, renormalize;
    dg_status st;
    CHECK(nargs == 8);
    f32 = is_dtype(arg[0], dtypes[F32]);
    CHECK((f32 || is_dtype(arg[0], dtypes[BF16])) && strided(arg[0], 2, &logits));
    CHECK(logits.stride[1] == 1 || logits.n[1] == 1);
    CHECK(is_dtype(arg[1], dtypes[I32]) && shape_of(arg[1], 2, &ids) && ids.n[0] == logits.n[0] && is_contiguous(arg[1]));
    CHECK(is_dtype(arg[2], dtypes[F32]) && shape_of(arg[2], 2, &weights) && is_contiguous(arg[2]));
    CHECK(weights.n[0] == ids.n[0] && weights.n[1] == ids.n[1]);
    CHECK(arg[3] == Py_None || (is_dtype(arg[3], dtypes[F32]) && shape_of(arg[3], 1, &bias) &&
                                bias.n[0] == logits.n[1] && is_contiguous(arg[3])));
    CHECK(logits.n[0] <= INT32_MAX && logits.n[1] <= INT32_MAX && ids.n[1] <= INT32_MAX);
    sigmoid = PyObject_IsTrue(arg[4]);
    renormalize = PyObject_IsTrue(arg[5]);
    scale = PyFloat_AsDouble(arg[6]);
    CHECK(!PyErr_Occurred() && placed(arg, 4) && stream_of(arg[7], arg[0], &stream));
    Py_BEGIN_ALLOW_THREADS
    st = ((RouteFn)fns[ROUTE])(logits.p, row_stride(&logits), f32 ? DG_LOGITS_F32 : DG_LOGITS_BF16, (const float *)bias.p,
                               (int32_t *)ids.p, (float *)weights.p, (int)logits.n[0], (int)logits.n[1], (int)ids.n[1],
                               sigmoid ? DG_SCORE_SIGMOID : DG_SCORE_SOFTMAX, renormalize, (float)scale, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
fail:
    return NULL;
}

static PyObject *layer(PyObject *self, PyObject *const *arg, Py_ssize_t nargs) {
    Tensor x, ids, weights, w1, w2, y, c = {{0, 0, 0}, {0, 0, 0}, NULL};
    PyObject *hold = NULL, *code;
    void *sf1, *sf2, *ws, *status, *stream;
    int64_t t, h, i, e, topk, ws_bytes, need, per, slice;
    int fp4;
    dg_status st;
    CHECK(nargs == 13);
    fp4 = PyObject_IsTrue(arg[0]);
    code = dtypes[fp4 ? U8 : FP8];
    per = fp4 ? 2 : 1;
    slice = fp4 ? 128 : 512;
    {
        PyObject *const tx = arg[1], *const tids = arg[2], *const tw = arg[3], *const t1 = arg[4], *const s1 = arg[5],
                        *const t2 = arg[6], *const s2 = arg[7], *const ty = arg[8], *const tc = arg[9];
        CHECK(strided(tx, 2, &x) && strided(ty, 2, &y) && is_dtype(tx, dtypes[BF16]) && is_dtype(ty, dtypes[BF16]));
        t = x.n[0];
        h = x.n[1];
        CHECK((x.stride[1] == 1 && y.stride[1] == 1) || h <= 1);
        CHECK(is_dtype(tids, dtypes[I32]) && shape_of(tids, 2, &ids) && ids.n[0] == t && is_contiguous(tids));
        topk = ids.n[1];
        CHECK(is_dtype(tw, dtypes[F32]) && shape_of(tw, 2, &weights) && is_contiguous(tw));
        CHECK(weights.n[0] == t && weights.n[1] == topk);
        CHECK(is_dtype(t1, code) && shape_of(t1, 3, &w1) && is_contiguous(t1));
        e = w1.n[0];
        i = w1.n[1] / 2;
        CHECK(w1.n[1] == 2 * i && w1.n[2] * per == h);
        CHECK(is_dtype(t2, code) && shape_of(t2, 3, &w2) && is_contiguous(t2));
        CHECK(w2.n[0] == e && w2.n[1] == h && w2.n[2] == i / per);
        CHECK(is_dtype(s1, dtypes[I32]) && is_contiguous(s1) && bytes_of(s1) >= e * ((h + slice - 1) / slice) * 2 * i * 4);
        CHECK(is_dtype(s2, dtypes[I32]) && is_contiguous(s2) && bytes_of(s2) >= e * ((i + slice - 1) / slice) * h * 4);
        CHECK(y.n[0] == t && y.n[1] == h);
        CHECK(tc == Py_None || (is_dtype(tc, dtypes[BF16]) && strided(tc, 2, &c) && c.n[0] == t && c.n[1] == h &&
                                (c.stride[1] == 1 || h <= 1)));
        CHECK(t <= INT32_MAX && h <= INT32_MAX && w1.n[1] <= INT32_MAX && e <= INT32_MAX && topk <= INT32_MAX);
        CHECK(pointer_of(s1, &sf1) && pointer_of(s2, &sf2) && status_of(arg[11], &status));
        need = ((LayerBytesFn)fns[LAYER_BYTES])((int)t, (int)topk, (int)h, (int)i, (int)e);
        PyObject *const on_device[] = {tx, tids, tw, t1, s1, t2, s2, ty, tc, arg[11]};
        CHECK(device_side(on_device, 10, arg[10], need, ty, arg[12], &hold, &ws, &ws_bytes, &stream));
    }
    Py_BEGIN_ALLOW_THREADS
    st = ((LayerFn)fns[fp4 ? LAYER_FP4 : LAYER_FP8])(
        x.p, row_stride(&x), (const int32_t *)ids.p, (const float *)weights.p, w1.p, sf1, w2.p, sf2, c.p,
        c.p ? row_stride(&c) : 0, y.p, row_stride(&y), (int)t, (int)h, (int)i, (int)e, (int)topk, ws, ws_bytes,
        (int32_t *)status, stream);
    Py_END_ALLOW_THREADS
    Py_XDECREF(hold);
    return PyLong_FromLong(st);
fail:
    Py_XDECREF(hold);
    return NULL;
}

/* A matrix, or (lead >= 0) `lead` of them, of this dtype and these sizes, with unit column stride: its
 * pointer and row stride in elements (of a single row: its length in whole 16s), the stride
 * from one matrix to the next. */
typedef struct {
    void *p;
    int64_t ld, batch;
} Matrix;

static int matrix_of(PyObject *t, PyObject *dtype, int64_t lead, int64_t rows, int64_t cols, Matrix *out) {
    Tensor x;
    const int d = lead >= 0 ? 1 : 0;
    out->p = NULL;
    out->ld = out->batch = 0;
    if (!is_dtype(t, dtype) || !strided(t, 2 + d, &x)) return 0;
    if ((d && x.n[0] != lead) || x.n[d] != rows || x.n[d + 1] != cols || (x.stride[d + 1] != 1 && cols > 1)) return 0;
    out->p = x.p;
    out->ld = rows > 1 ? x.stride[d] : (cols + 15) / 16 * 16;
    out->batch = d && lead > 1 ? x.stride[0] : 0;
    return 1;
}

/* Not given, or a matrix. */
static int matrix_or_none(PyObject *t, PyObject *dtype, int64_t lead, int64_t rows, int64_t cols, Matrix *out) {
    out->p = NULL;
    out->ld = out->batch = 0;
    return t == Py_None || matrix_of(t, dtype, lead, rows, cols, out);
}

/* Dense int32 words, this many. */
static int words_of(PyObject *t, int64_t count, void **out) {
    return is_dtype(t, dtypes[I32]) && is_contiguous(t) && bytes_of(t) == 4 * count && pointer_of(t, out);
}

static int64_t slices_of(int64_t k) { return (k + 511) / 512; }
static int64_t align4_of(int64_t n) { return (n + 3) / 4 * 4; }

/* The last dimensions of a 2-D or 3-D tensor; lead is -1 where it is 2-D. */
static int sizes_of(PyObject *t, int64_t *lead, int64_t *rows, int64_t *cols) {
    PyObject *shape = PyObject_GetAttr(t, s_shape);
    int64_t n[3];
    int d;
    if (!shape || !PyTuple_Check(shape)) {
        Py_XDECREF(shape);
        return 0;
    }
    d = PyTuple_GET_SIZE(shape) == 3;
    if (!dims_of(shape, 2 + d, n)) return 0;
    *lead = d ? n[0] : -1;
    *rows = n[d];
    *cols = n[d + 1];
    return *lead <= INT32_MAX && *rows <= INT32_MAX && *cols <= INT32_MAX;
}

/* gated(a, sfa, b, sfb, layout or None, h, hq, sfh, gu, status, stream) */
static PyObject *gated(PyObject *self, PyObject *const *arg, Py_ssize_t nargs) {
    Matrix a, b, h, hq, gu;
    void *sfa, *sfb, *sfh = NULL, *layout = NULL, *status, *stream;
    int64_t m, k, i, e, none;
    int grouped;
    dg_status st;
    CHECK(nargs == 11);
    grouped = arg[4] != Py_None;
    CHECK(sizes_of(arg[0], &none, &m, &k) && none < 0 && sizes_of(arg[2], &e, &i, &none) && (e >= 0) == grouped);
    CHECK(i % 2 == 0);
    i /= 2;
    CHECK(matrix_of(arg[0], dtypes[FP8], -1, m, k, &a) && matrix_of(arg[2], dtypes[FP8], e, 2 * i, k, &b));
    CHECK(e <= 1 || b.batch == 2 * i * b.ld);   /* experts follow one another */
    CHECK(words_of(arg[1], slices_of(k) * align4_of(m), &sfa));
    CHECK(words_of(arg[3], (grouped ? e : 1) * slices_of(k) * align4_of(2 * i), &sfb));
    CHECK((arg[5] == Py_None) != (arg[6] == Py_None));   /* exactly one of h and hq */
    CHECK(matrix_or_none(arg[5], dtypes[BF16], -1, m, i, &h) && matrix_or_none(arg[6], dtypes[FP8], -1, m, i, &hq));
    CHECK(matrix_or_none(arg[8], dtypes[BF16], -1, m, 2 * i, &gu));
    CHECK(arg[6] == Py_None || words_of(arg[7], slices_of(i) * align4_of(m), &sfh));
    CHECK(!grouped || words_of(arg[4], m, &layout));
    CHECK(status_of(arg[9], &status) && placed(arg, 7) && placed(arg + 8, 2));
    CHECK((arg[6] == Py_None || placed(arg + 7, 1)) && stream_of(arg[10], arg[0], &stream));
    Py_BEGIN_ALLOW_THREADS
    st = grouped ? ((GatedGroupedFn)fns[GATED_GROUPED])(a.p, a.ld, sfa, b.p, b.ld, sfb, gu.p, gu.ld, h.p, h.ld, hq.p,
                                                        hq.ld, sfh, (const int32_t *)layout, (int)m, (int)i, (int)k,
                                                        (int)e, (int32_t *)status, stream)
                 : ((GatedFn)fns[GATED])(a.p, a.ld, sfa, b.p, b.ld, sfb, gu.p, gu.ld, h.p, h.ld, hq.p, hq.ld, sfh,
                                         (int)m, (int)i, (int)k, (int32_t *)status, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
fail:
    return NULL;
}

/* gated_backward(dy, sfdy, w2, sfw2, layout or None, gu, dgu, h, status, stream) */
static PyObject *gated_backward(PyObject *self, PyObject *const *arg, Py_ssize_t nargs) {
    Matrix dy, w2, gu, dgu, h;
    void *sfdy, *sfw2, *layout = NULL, *status, *stream;
    int64_t m, k, i, e, rows, none;
    int grouped;
    dg_status st;
    CHECK(nargs == 10);
    grouped = arg[4] != Py_None;
    CHECK(sizes_of(arg[0], &none, &m, &k) && none < 0 && sizes_of(arg[2], &e, &rows, &i) && (e >= 0) == grouped);
    CHECK(rows == k && i <= INT32_MAX / 2);
    CHECK(matrix_of(arg[0], dtypes[FP8], -1, m, k, &dy) && matrix_of(arg[2], dtypes[FP8], e, k, i, &w2));
    CHECK(e <= 1 || w2.batch == k * w2.ld);   /* experts follow one another */
    CHECK(words_of(arg[1], slices_of(k) * align4_of(m), &sfdy));
    CHECK(words_of(arg[3], (grouped ? e : 1) * slices_of(k) * align4_of(i), &sfw2));
    CHECK(matrix_of(arg[5], dtypes[BF16], -1, m, 2 * i, &gu) && matrix_of(arg[6], dtypes[BF16], -1, m, 2 * i, &dgu));
    CHECK(matrix_or_none(arg[7], dtypes[BF16], -1, m, i, &h));
    CHECK(!grouped || words_of(arg[4], m, &layout));
    CHECK(status_of(arg[8], &status) && placed(arg, 9) && stream_of(arg[9], arg[0], &stream));
    Py_BEGIN_ALLOW_THREADS
    st = grouped ? ((BackwardGroupedFn)fns[BACKWARD_GROUPED])(dy.p, dy.ld, sfdy, w2.p, w2.ld, sfw2, gu.p, gu.ld, dgu.p,
                                                              dgu.ld, h.p, h.ld, (const int32_t *)layout, (int)m, (int)i,
                                                              (int)k, (int)e, (int32_t *)status, stream)
                 : ((BackwardFn)fns[BACKWARD])(dy.p, dy.ld, sfdy, w2.p, w2.ld, sfw2, gu.p, gu.ld, dgu.p, dgu.ld, h.p,
                                               h.ld, (int)m, (int)i, (int)k, (int32_t *)status, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
fail:
    return NULL;
}

/* quantize(x, q, sf, qk, sfk, ks or None, stream) */
static PyObject *quantize(PyObject *self, PyObject *const *arg, Py_ssize_t nargs) {
    Matrix x, q, qk;
    PyObject *list = NULL;
    void *sf = NULL, *sfk = NULL, *stream;
    int64_t r, c, none, packed;
    int ks[256], groups = 0, f32, j;
    dg_status st;
    CHECK(nargs == 7);
    f32 = is_dtype(arg[0], dtypes[F32]);
    CHECK(sizes_of(arg[0], &none, &r, &c) && none < 0 && matrix_of(arg[0], dtypes[f32 ? F32 : BF16], -1, r, c, &x));
    CHECK(arg[1] != Py_None || arg[3] != Py_None);   /* q or qk */
    CHECK(matrix_or_none(arg[1], dtypes[FP8], -1, r, c, &q) && matrix_or_none(arg[3], dtypes[FP8], -1, r, c, &qk));
    CHECK(arg[1] == Py_None || words_of(arg[2], slices_of(c) * align4_of(r), &sf));
    packed = slices_of(r) * align4_of(c);
    if (arg[5] != Py_None) {
        list = PySequence_Fast(arg[5], "ks is a list of group sizes");
        CHECK(list && PySequence_Fast_GET_SIZE(list) <= 255);
        groups = (int)PySequence_Fast_GET_SIZE(list);
        for (j = 0; j < groups; ++j) {
            const int64_t k = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(list, j));
            CHECK(!(k == -1 && PyErr_Occurred()) && k >= 0 && k <= INT32_MAX && k % 128 == 0);
            ks[j] = (int)k;
        }
        packed = ((PackedRowsFn)fns[PACKED_ROWS])(ks, groups) * c;
        CHECK(packed >= 0);
    }
    CHECK(arg[3] == Py_None || words_of(arg[4], packed, &sfk));
    CHECK(placed(arg, 2) && placed(arg + 3, 1) && (!sf || placed(arg + 2, 1)) && (!sfk || placed(arg + 4, 1)));
    CHECK(stream_of(arg[6], arg[0], &stream));
    Py_BEGIN_ALLOW_THREADS
    st = ((QuantizeFn)fns[QUANTIZE])(x.p, f32 ? DG_VALUES_F32 : DG_VALUES_BF16, x.ld, q.p, q.ld, sf, qk.p, qk.ld, sfk,
                                     (int)r, (int)c, list ? ks : NULL, groups, stream);
    Py_END_ALLOW_THREADS
    Py_XDECREF(list);
    return PyLong_FromLong(st);
fail:
    Py_XDECREF(list);
    return NULL;
}

/* quantize_blocks(x, q, sf, sft, stream) */
static PyObject *quantize_blocks(PyObject *self, PyObject *const *arg, Py_ssize_t nargs) {
    Matrix x, q;
    void *sf = NULL, *sft = NULL, *stream;
    int64_t lead, r, c, b;
    int f32;
    dg_status st;
    CHECK(nargs == 5);
    f32 = is_dtype(arg[0], dtypes[F32]);
    CHECK(sizes_of(arg[0], &lead, &r, &c) && matrix_of(arg[0], dtypes[f32 ? F32 : BF16], lead, r, c, &x));
    CHECK(matrix_of(arg[1], dtypes[FP8], lead, r, c, &q) && (arg[2] != Py_None || arg[3] != Py_None));   /* sf or sft */
    b = lead < 0 ? 1 : lead;
    CHECK(arg[2] == Py_None || words_of(arg[2], b * slices_of(c) * align4_of(r), &sf));
    CHECK(arg[3] == Py_None || words_of(arg[3], b * slices_of(r) * align4_of(c), &sft));
    CHECK(placed(arg, 4) && stream_of(arg[4], arg[0], &stream));
    Py_BEGIN_ALLOW_THREADS
    st = ((BlocksFn)fns[BLOCKS])(x.p, f32 ? DG_VALUES_F32 : DG_VALUES_BF16, x.ld, x.batch, q.p, q.ld, q.batch, sf, sft,
                                 (int)b, (int)r, (int)c, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
fail:
    return NULL;
}

/* newton_schulz(g, out, steps, a, b, c, eps, workspace, status, stream) */
static PyObject *newton_schulz(PyObject *self, PyObject *const *arg, Py_ssize_t nargs) {
    Matrix g, out;
    PyObject *hold = NULL;
    void *ws, *status, *stream;
    int64_t lead, r, c, lo, hi, batch, steps, need, ws_bytes;
    double coef[4];
    int f32, j;
    dg_status st;
    CHECK(nargs == 10);
    f32 = is_dtype(arg[0], dtypes[F32]);
    CHECK(sizes_of(arg[0], &lead, &r, &c) && matrix_of(arg[0], dtypes[f32 ? F32 : BF16], lead, r, c, &g));
    CHECK(matrix_of(arg[1], dtypes[BF16], lead, r, c, &out));
    steps = PyLong_AsLongLong(arg[2]);
    for (j = 0; j < 4; ++j) coef[j] = PyFloat_AsDouble(arg[3 + j]);
    CHECK(!PyErr_Occurred() && steps >= INT32_MIN && steps <= INT32_MAX);
    batch = lead < 0 ? 1 : lead;
    CHECK(status_of(arg[8], &status));
    need = ((SchulzBytesFn)fns[SCHULZ_BYTES])((int)batch, (int)r, (int)c);
    lo = r < c ? r : c;
    hi = r < c ? c : r;
    /* (refused; the last: more tiles than the kernels count) */
    if (steps < 1 || steps > 1000 || !(coef[3] >= 0) ||
        (need >= 0 && 6 * steps * batch * ((lo + 255) / 256) * ((hi + 63) / 64) > INT32_MAX))
        need = -1;
    PyObject *const on_device[] = {arg[0], arg[1], arg[8]};
    CHECK(device_side(on_device, 3, arg[7], need, arg[0], arg[9], &hold, &ws, &ws_bytes, &stream));
    Py_BEGIN_ALLOW_THREADS
    st = ((SchulzFn)fns[SCHULZ])(g.p, f32 ? DG_VALUES_F32 : DG_VALUES_BF16, g.ld, g.batch, out.p, out.ld, out.batch,
                                 (int)batch, (int)r, (int)c, (int)steps, (float)coef[0], (float)coef[1], (float)coef[2],
                                 (float)coef[3], ws, ws_bytes, (int32_t *)status, stream);
    Py_END_ALLOW_THREADS
    Py_XDECREF(hold);
    return PyLong_FromLong(st);
fail:
    Py_XDECREF(hold);
    return NULL;
}

/* setup(addresses of the entry points, dtypes, raw stream of a device, current device, workspace maker) */
static PyObject *setup(PyObject *self, PyObject *args) {
    PyObject *addresses, *types;
    int i;
    if (!PyArg_ParseTuple(args, "O!O!OOO", &PyTuple_Type, &addresses, &PyTuple_Type, &types, &raw_stream, &current_device,
                          &make_workspace))
        return NULL;
    CHECK(PyTuple_GET_SIZE(addresses) == FNS && PyTuple_GET_SIZE(types) == DTYPES);
    for (i = 0; i < FNS; ++i) {
        fns[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(addresses, i));
        CHECK(fns[i]);
    }
    for (i = 0; i < DTYPES; ++i) Py_INCREF(dtypes[i] = PyTuple_GET_ITEM(types, i));
    Py_INCREF(raw_stream);
    Py_INCREF(current_device);
    Py_INCREF(make_workspace);
    Py_RETURN_NONE;
fail:
    return NULL;
}

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, NULL},
    {"gemv", (PyCFunction)(void (*)(void))gemv, METH_FASTCALL, NULL},
    {"route", (PyCFunction)(void (*)(void))route, METH_FASTCALL, NULL},
    {"layer", (PyCFunction)(void (*)(void))layer, METH_FASTCALL, NULL},
    {"gated", (PyCFunction)(void (*)(void))gated, METH_FASTCALL, NULL},
    {"gated_backward", (PyCFunction)(void (*)(void))gated_backward, METH_FASTCALL, NULL},
    {"quantize", (PyCFunction)(void (*)(void))quantize, METH_FASTCALL, NULL},
    {"quantize_blocks", (PyCFunction)(void (*)(void))quantize_blocks, METH_FASTCALL, NULL},
    {"newton_schulz", (PyCFunction)(void (*)(void))newton_schulz, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "dg_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit_dg_marshal(void) {
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_stride = PyUnicode_InternFromString("stride");
    s_shape = PyUnicode_InternFromString("shape");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_nbytes = PyUnicode_InternFromString("nbytes");
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    return PyModule_Create(&module);
}
