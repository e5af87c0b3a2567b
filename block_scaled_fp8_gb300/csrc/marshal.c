/* Marshalling of the decode calls (few-row products, routing, the MoE layer) from torch tensors
 * to the C ABI, for binding.py.  Such a call takes a few microseconds on the device, and its
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

enum { GEMV_FP4, GEMV_FP8, GEMV_FP4_F32, GEMV_FP8_F32, ROUTE, LAYER_FP4, LAYER_FP8, GEMV_BYTES, LAYER_BYTES, FNS };
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
