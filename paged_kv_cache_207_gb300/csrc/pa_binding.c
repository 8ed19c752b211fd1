/*
 * pa_binding.c -- the quick way through the Python bindings of the calls that a decode step
 * makes once per layer (rotary append, windowed decode and prefill attention).
 *
 * A short step waits for the host, not for the GPU: checking a dozen tensors from Python and
 * marshalling two dozen arguments through ctypes costs about twice the launch itself (on the
 * Grace host of a GB300, per call: decode 9.0 us in Python, 4.1 us of it the call).  These
 * functions make the same checks of a call whose arguments are all as they should be, on the
 * current device and stream, and call the library.  Anything else -- a tensor of another type,
 * shape, device or layout, an explicit stream, an object that is no tensor -- returns -1 and
 * does nothing: the Python binding then looks closer, raises what there is to raise, or makes
 * the call itself.  Nothing is kept between calls.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "pa.h"

typedef pa_status (*rope_fn)(void*, void*, void*, const void*, const void*, const void*, int64_t, int64_t, int64_t,
                             int64_t, const double*, int32_t, int32_t, const int32_t*, int32_t, const int32_t*,
                             const int32_t*, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, pa_dtype, int32_t*,
                             void*);
typedef pa_status (*decode_fn)(void*, const void*, const void*, const void*, const int32_t*, const int32_t*, int32_t,
                               int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, float, pa_dtype, int32_t*,
                               void*);
typedef pa_status (*prefill_fn)(void*, const void*, const void*, const void*, const int32_t*, int32_t, const int32_t*,
                                const int32_t*, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t,
                                int32_t, float, pa_dtype, int32_t*, void*);

static rope_fn call_rope;
static decode_fn call_decode;
static prefill_fn call_prefill;
static PyTypeObject* tensor_type;
static PyObject *f32, *bf16, *u8, *i32, *f64;                  /* torch dtypes (one object each) */
static PyObject *current_device, *raw_stream;                  /* torch functions */
static PyObject *n_dtype, *n_shape, *n_get_device, *n_is_contiguous, *n_data_ptr, *n_stride;

enum { MAX_DIMS = 5 };
typedef struct {
    PyObject* dtype;
    int dims;
    int64_t shape[MAX_DIMS], stride[MAX_DIMS];
    long device;
    void* ptr;
} Info;

static PyObject* method(PyObject* t, PyObject* name) {
    PyObject* args[1] = {t};
    return PyObject_VectorcallMethod(name, args, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, NULL);
}

static int long_of(PyObject* v, int64_t* out) {                /* takes the reference */
    if (!v) return -1;
    *out = PyLong_AsLongLong(v);
    Py_DECREF(v);
    return *out == -1 && PyErr_Occurred() ? -1 : 0;
}

static int longs_of(PyObject* v, int* count, int64_t* out) {   /* a tuple of sizes; takes the reference */
    if (!v) return -1;
    int ok = PyTuple_Check(v) && PyTuple_GET_SIZE(v) <= MAX_DIMS ? 0 : -1;
    if (ok == 0) {
        *count = (int)PyTuple_GET_SIZE(v);
        for (int i = 0; i < *count && ok == 0; ++i) {
            out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(v, i));
            if ((out[i] == -1 && PyErr_Occurred()) || out[i] > INT64_MAX / 64) ok = -1;
        }
    }
    Py_DECREF(v);
    return ok;
}

/* What a call needs to know of a tensor; with `strided`, its strides in place of contiguity. */
static int look(PyObject* t, Info* x, int strided) {
    if (!tensor_type || !PyObject_TypeCheck(t, tensor_type)) return -1;
    PyObject* v = PyObject_GetAttr(t, n_dtype);
    if (!v) return -1;
    x->dtype = v;                                              /* only compared: dtypes live as long as torch */
    Py_DECREF(v);
    int64_t n;
    if (longs_of(PyObject_GetAttr(t, n_shape), &x->dims, x->shape) < 0) return -1;
    if (long_of(method(t, n_get_device), &n) < 0) return -1;
    x->device = (long)n;
    if (strided) {
        int dims;
        if (longs_of(method(t, n_stride), &dims, x->stride) < 0) return -1;
    } else {
        v = method(t, n_is_contiguous);
        if (!v) return -1;
        const int yes = v == Py_True;
        Py_DECREF(v);
        if (!yes) return -1;
    }
    if (long_of(method(t, n_data_ptr), &n) < 0) return -1;
    x->ptr = (void*)(intptr_t)n;
    return 0;
}

static int small(int64_t v) { return v >= 0 && v <= INT32_MAX; }

static int is_vector(const Info* x, PyObject* dtype, int64_t n, long device) {
    return x->dtype == dtype && x->dims == 1 && x->shape[0] == n && x->device == device;
}

typedef struct {
    Info k, v;
    int32_t blocks, heads, dim;
    pa_dtype code;
    PyObject* rows;                                            /* type of rows, q and out */
} Pools;

static int look_pools(PyObject* k, PyObject* v, int64_t kind, Pools* p) {
    if (look(k, &p->k, 0) < 0 || look(v, &p->v, 0) < 0) return -1;
    const Info* x = &p->k;
    int64_t dim;
    if (kind == PA_FP8_E4M3 || kind == PA_FP4_E2M1) {
        if (x->dtype != u8 || x->dims != 3) return -1;
        if (kind == PA_FP8_E4M3 ? (x->shape[2] - 64) % 16 != 0 : x->shape[2] % 17 != 0) return -1;
        dim = kind == PA_FP8_E4M3 ? (x->shape[2] - 64) / 16 : x->shape[2] * 2 / 17;
        p->code = (pa_dtype)kind;
        p->rows = bf16;
    } else {
        if (x->dims != 5 || x->shape[3] != PA_BLOCK_SIZE || (x->dtype != f32 && x->dtype != bf16)) return -1;
        dim = x->shape[2] * x->shape[4];
        p->code = x->dtype == f32 ? PA_F32 : PA_BF16;
        p->rows = x->dtype;
    }
    if (p->v.dtype != x->dtype || p->v.dims != x->dims || p->v.device != x->device || x->device < 0) return -1;
    for (int i = 0; i < x->dims; ++i)
        if (p->v.shape[i] != x->shape[i]) return -1;
    if (!small(x->shape[0]) || !small(x->shape[1]) || !small(dim)) return -1;
    p->blocks = (int32_t)x->shape[0];
    p->heads = (int32_t)x->shape[1];
    p->dim = (int32_t)dim;
    return 0;
}

/* The error flag (None: NULL), the current stream of the pools' device if that is the current one. */
static int look_rest(PyObject* flag, PyObject* stream, long device, int32_t** err, void** raw) {
    if (stream != Py_None) return -1;
    *err = NULL;
    if (flag != Py_None) {
        Info x;
        if (look(flag, &x, 0) < 0 || x.dtype != i32 || x.device != device) return -1;
        *err = (int32_t*)x.ptr;
    }
    int64_t n;
    if (long_of(PyObject_CallNoArgs(current_device), &n) < 0 || n != device) return -1;
    PyObject* d = PyLong_FromLong(device);
    if (!d) return -1;
    PyObject* v = PyObject_CallOneArg(raw_stream, d);
    Py_DECREF(d);
    if (long_of(v, &n) < 0) return -1;
    *raw = (void*)(intptr_t)n;
    return 0;
}

/* An int, with anything past int32 as the largest. */
static int bound_of(PyObject* v, int32_t* out) {
    if (!PyLong_CheckExact(v)) return -1;
    int over;
    const long long n = PyLong_AsLongLongAndOverflow(v, &over);
    if (over < 0 || (over == 0 && n < INT32_MIN)) return -1;
    *out = over > 0 || n > INT32_MAX ? INT32_MAX : (int32_t)n;
    return 0;
}

static PyObject* closer(void) {
    PyErr_Clear();
    return PyLong_FromLong(-1);
}

/* decode_window(kind, out, q, k_pool, v_pool, tables, lens, scale, window, sinks, flag, stream) */
static PyObject* decode_window(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Pools p;
    Info out, q, tables, lens;
    int32_t window, sinks, *err;
    void* raw;
    if (n != 12 || look_pools(a[3], a[4], PyLong_AsLong(a[0]), &p) < 0) return closer();
    const long dev = p.k.device;
    if (look(a[1], &out, 0) < 0 || look(a[2], &q, 0) < 0 || look(a[5], &tables, 0) < 0 || look(a[6], &lens, 0) < 0)
        return closer();
    if (q.dtype != p.rows || out.dtype != p.rows || q.dims != 3 || out.dims != 3 || q.device != dev || out.device != dev)
        return closer();
    for (int i = 0; i < 3; ++i)
        if (out.shape[i] != q.shape[i] || !small(q.shape[i])) return closer();
    if (q.shape[2] != p.dim || tables.dtype != i32 || tables.dims != 2 || tables.shape[0] != q.shape[0] ||
        !small(tables.shape[1]) || tables.device != dev || !is_vector(&lens, i32, q.shape[0], dev))
        return closer();
    const double scale = PyFloat_AsDouble(a[7]);
    if (scale == -1.0 && PyErr_Occurred()) return closer();
    if (bound_of(a[8], &window) < 0 || bound_of(a[9], &sinks) < 0 || look_rest(a[10], a[11], dev, &err, &raw) < 0)
        return closer();
    pa_status s;
    Py_BEGIN_ALLOW_THREADS
    s = call_decode(out.ptr, q.ptr, p.k.ptr, p.v.ptr, tables.ptr, lens.ptr, (int32_t)q.shape[0], (int32_t)q.shape[1],
                    p.heads, p.dim, (int32_t)tables.shape[1], p.blocks, window, sinks, (float)scale, p.code, err, raw);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(s);
}

/* prefill_window(out, q, k_pool, v_pool, tables, start, cu, scale, max_chunk, window, sinks, flag, stream) */
static PyObject* prefill_window(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Pools p;
    Info out, q, tables, start, cu;
    int32_t chunk, window, sinks, *err;
    void* raw;
    if (n != 13 || look_pools(a[2], a[3], PA_BF16, &p) < 0) return closer();
    const long dev = p.k.device;
    if (look(a[0], &out, 0) < 0 || look(a[1], &q, 0) < 0 || look(a[4], &tables, 0) < 0 || look(a[5], &start, 0) < 0 ||
        look(a[6], &cu, 0) < 0)
        return closer();
    if (q.dtype != p.rows || out.dtype != p.rows || q.dims != 3 || out.dims != 3 || q.device != dev || out.device != dev)
        return closer();
    for (int i = 0; i < 3; ++i)
        if (out.shape[i] != q.shape[i] || !small(q.shape[i])) return closer();
    if (q.shape[2] != p.dim || tables.dtype != i32 || tables.dims != 2 || !small(tables.shape[0]) ||
        !small(tables.shape[1]) || tables.device != dev || !is_vector(&start, i32, tables.shape[0], dev) ||
        !is_vector(&cu, i32, tables.shape[0] + 1, dev))
        return closer();
    const double scale = PyFloat_AsDouble(a[7]);
    if (scale == -1.0 && PyErr_Occurred()) return closer();
    if (bound_of(a[8], &chunk) < 0 || bound_of(a[9], &window) < 0 || bound_of(a[10], &sinks) < 0 ||
        look_rest(a[11], a[12], dev, &err, &raw) < 0)
        return closer();
    pa_status s;
    Py_BEGIN_ALLOW_THREADS
    s = call_prefill(out.ptr, q.ptr, p.k.ptr, p.v.ptr, tables.ptr, (int32_t)tables.shape[1], start.ptr, cu.ptr,
                     (int32_t)tables.shape[0], (int32_t)q.shape[0], chunk, (int32_t)q.shape[1], p.heads, p.dim, p.blocks,
                     window, sinks, (float)scale, p.code, err, raw);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(s);
}

/* Rows [n][heads][dim] whose rows may lie apart: a row's heads are contiguous. */
static int look_rows(PyObject* t, const Pools* p, int64_t n, int64_t heads, Info* x) {
    if (look(t, x, 1) < 0 || x->dtype != p->rows || x->dims != 3 || x->device != p->k.device) return -1;
    if ((n >= 0 && x->shape[0] != n) || (heads >= 0 && x->shape[1] != heads) || x->shape[2] != p->dim) return -1;
    if (!small(x->shape[0]) || !small(x->shape[1])) return -1;
    if (x->stride[2] != 1 || x->stride[1] != p->dim) return -1;
    if (x->shape[0] <= 1) x->stride[0] = x->shape[1] * p->dim;
    return 0;
}

/* rope_append(kind, k_pool, v_pool, q_out, q, k_new, v_new, inv_freq, tables, start, cu, interleaved, flag, stream) */
static PyObject* rope_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Pools p;
    Info qo, q, k, v, freq, tables, start, cu;
    int32_t* err;
    void* raw;
    if (n != 14 || look_pools(a[1], a[2], PyLong_AsLong(a[0]), &p) < 0) return closer();
    const long dev = p.k.device;
    if (look_rows(a[5], &p, -1, p.heads, &k) < 0 || look_rows(a[6], &p, k.shape[0], p.heads, &v) < 0) return closer();
    if (a[4] == Py_None && a[3] == Py_None) {
        q.ptr = qo.ptr = NULL;
        q.shape[1] = q.stride[0] = qo.stride[0] = 0;
    } else if (look_rows(a[4], &p, k.shape[0], -1, &q) < 0 || look_rows(a[3], &p, k.shape[0], q.shape[1], &qo) < 0) {
        return closer();
    }
    if (look(a[7], &freq, 0) < 0 || look(a[8], &tables, 0) < 0 || look(a[9], &start, 0) < 0 || look(a[10], &cu, 0) < 0)
        return closer();
    if (freq.dims != 1 || freq.shape[0] > 1 << 20 || !is_vector(&freq, f64, freq.shape[0], dev) || tables.dtype != i32 ||
        tables.dims != 2 || !small(tables.shape[0]) || !small(tables.shape[1]) || tables.device != dev ||
        !is_vector(&start, i32, tables.shape[0], dev) || !is_vector(&cu, i32, tables.shape[0] + 1, dev))
        return closer();
    const int interleaved = PyObject_IsTrue(a[11]);
    if (interleaved < 0 || look_rest(a[12], a[13], dev, &err, &raw) < 0) return closer();
    pa_status s;
    Py_BEGIN_ALLOW_THREADS
    s = call_rope(p.k.ptr, p.v.ptr, qo.ptr, q.ptr, k.ptr, v.ptr, qo.stride[0], q.stride[0], k.stride[0], v.stride[0],
                  freq.ptr, (int32_t)(2 * freq.shape[0]), interleaved, tables.ptr, (int32_t)tables.shape[1], start.ptr,
                  cu.ptr, (int32_t)tables.shape[0], (int32_t)k.shape[0], p.blocks, (int32_t)q.shape[1], p.heads, p.dim,
                  p.code, err, raw);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(s);
}

static PyObject* keep(PyObject* v) {
    Py_INCREF(v);
    return v;
}

/* bind(rope, decode, prefill, Tensor, float32, bfloat16, uint8, int32, float64, current_device, raw_stream):
 * the addresses of the library's functions and torch's objects, once, before any other call. */
static PyObject* bind(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (n != 11 || !PyType_Check(a[3])) {
        PyErr_SetString(PyExc_TypeError, "bind: three addresses, the tensor type, five dtypes, two functions");
        return NULL;
    }
    void* at[3];
    for (int i = 0; i < 3; ++i) {
        at[i] = PyLong_AsVoidPtr(a[i]);
        if (!at[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null address");
            return NULL;
        }
    }
    if (!tensor_type) {
        call_rope = (rope_fn)at[0];
        call_decode = (decode_fn)at[1];
        call_prefill = (prefill_fn)at[2];
        f32 = keep(a[4]);
        bf16 = keep(a[5]);
        u8 = keep(a[6]);
        i32 = keep(a[7]);
        f64 = keep(a[8]);
        current_device = keep(a[9]);
        raw_stream = keep(a[10]);
        tensor_type = (PyTypeObject*)keep(a[3]);
    }
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, NULL},
    {"rope_append", (PyCFunction)(void (*)(void))rope_append, METH_FASTCALL, NULL},
    {"decode_window", (PyCFunction)(void (*)(void))decode_window, METH_FASTCALL, NULL},
    {"prefill_window", (PyCFunction)(void (*)(void))prefill_window, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_quick", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__quick(void) {
    n_dtype = PyUnicode_InternFromString("dtype");
    n_shape = PyUnicode_InternFromString("shape");
    n_get_device = PyUnicode_InternFromString("get_device");
    n_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    n_data_ptr = PyUnicode_InternFromString("data_ptr");
    n_stride = PyUnicode_InternFromString("stride");
    if (!n_dtype || !n_shape || !n_get_device || !n_is_contiguous || !n_data_ptr || !n_stride) return NULL;
    return PyModule_Create(&module);
}
