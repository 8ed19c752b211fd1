/*
 * pa_binding.cpp -- the quick way through the Python bindings of the calls that a decode step
 * makes once per layer (rotary append, windowed decode and prefill attention).
 *
 * A short step waits for the host, not for the GPU: checking a dozen tensors from Python and
 * marshalling two dozen arguments through ctypes costs about twice the launch itself.  These
 * functions make the same checks of a call whose arguments are all as they should be, on the
 * tensors themselves, on the current device and stream, and call the library (on the Grace host
 * of a GB300, a decode call: 2.8 us, 5.1 when the tensors are asked through Python's methods,
 * 10.5 in Python; a rotary append of ten tensors 2.8 us, 6.5).  Anything else -- a tensor of
 * another type, shape, device or layout, a subclass, an explicit stream, an object that is no
 * tensor -- returns -1 and does nothing: the Python binding then looks closer, raises what there
 * is to raise, or makes the call itself.  Nothing is kept between calls.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "pa.h"

namespace {

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

rope_fn call_rope;
decode_fn call_decode;
prefill_fn call_prefill;

struct Address {
    void* at;
    template <typename T>
    operator T*() const { return static_cast<T*>(at); }
};

constexpr int MAX_DIMS = 5;
struct Info {
    at::ScalarType dtype;
    int dims;
    int64_t shape[MAX_DIMS], stride[MAX_DIMS];
    long device;                                               /* -1: not on a GPU */
    Address ptr;
};

/* What a call needs to know of a tensor; with `strided`, its strides in place of contiguity. */
int look(PyObject* t, Info* x, bool strided) {
    if (!THPVariable_CheckExact(t)) return -1;
    const at::Tensor& y = THPVariable_Unpack(t);
    if (!y.defined() || y.layout() != at::kStrided || y.dim() > MAX_DIMS || (!strided && !y.is_contiguous())) return -1;
    x->dtype = y.scalar_type();
    x->dims = (int)y.dim();
    for (int i = 0; i < x->dims; ++i) {
        x->shape[i] = y.size(i);
        x->stride[i] = y.stride(i);
        if (x->shape[i] > INT64_MAX / 64) return -1;
    }
    x->device = y.is_cuda() ? y.get_device() : -1;
    x->ptr.at = y.data_ptr();
    return 0;
}

bool small(int64_t v) { return v >= 0 && v <= INT32_MAX; }

bool is_vector(const Info* x, at::ScalarType dtype, int64_t n, long device) {
    return x->dtype == dtype && x->dims == 1 && x->shape[0] == n && x->device == device;
}

struct Pools {
    Info k, v;
    int32_t blocks, heads, dim;
    pa_dtype code;
    at::ScalarType rows;                                       /* type of rows, q and out */
};

int look_pools(PyObject* k, PyObject* v, int64_t kind, Pools* p) {
    if (look(k, &p->k, false) < 0 || look(v, &p->v, false) < 0) return -1;
    const Info* x = &p->k;
    int64_t dim;
    if (kind == PA_FP8_E4M3 || kind == PA_FP4_E2M1) {
        if (x->dtype != at::kByte || x->dims != 3) return -1;
        if (kind == PA_FP8_E4M3 ? (x->shape[2] - 64) % 16 != 0 : x->shape[2] % 17 != 0) return -1;
        dim = kind == PA_FP8_E4M3 ? (x->shape[2] - 64) / 16 : x->shape[2] * 2 / 17;
        p->code = (pa_dtype)kind;
        p->rows = at::kBFloat16;
    } else {
        if (x->dims != 5 || x->shape[3] != PA_BLOCK_SIZE || (x->dtype != at::kFloat && x->dtype != at::kBFloat16)) return -1;
        dim = x->shape[2] * x->shape[4];
        p->code = x->dtype == at::kFloat ? PA_F32 : PA_BF16;
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

/* The error flag (None: nullptr), the current stream of the pools' device if that is the current one. */
int look_rest(PyObject* flag, PyObject* stream, long device, int32_t** err, void** raw) {
    if (stream != Py_None) return -1;
    *err = nullptr;
    if (flag != Py_None) {
        Info x;
        if (look(flag, &x, false) < 0 || x.dtype != at::kInt || x.device != device) return -1;
        *err = x.ptr;
    }
    if (c10::cuda::current_device() != device) return -1;
    *raw = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    return 0;
}

/* An int, with anything past int32 as the largest. */
int bound_of(PyObject* v, int32_t* out) {
    if (!PyLong_CheckExact(v)) return -1;
    int over;
    const long long n = PyLong_AsLongLongAndOverflow(v, &over);
    if (over < 0 || (over == 0 && n < INT32_MIN)) return -1;
    *out = over > 0 || n > INT32_MAX ? INT32_MAX : (int32_t)n;
    return 0;
}

PyObject* closer(void) {
    PyErr_Clear();
    return PyLong_FromLong(-1);
}

/* decode_window(kind, out, q, k_pool, v_pool, tables, lens, scale, window, sinks, flag, stream) */
PyObject* decode_window(PyObject* const* a, Py_ssize_t n) {
    Pools p;
    Info out, q, tables, lens;
    int32_t window, sinks, *err;
    void* raw;
    if (n != 12 || look_pools(a[3], a[4], PyLong_AsLong(a[0]), &p) < 0) return closer();
    const long dev = p.k.device;
    if (look(a[1], &out, false) < 0 || look(a[2], &q, false) < 0 || look(a[5], &tables, false) < 0 || look(a[6], &lens, false) < 0)
        return closer();
    if (q.dtype != p.rows || out.dtype != p.rows || q.dims != 3 || out.dims != 3 || q.device != dev || out.device != dev)
        return closer();
    for (int i = 0; i < 3; ++i)
        if (out.shape[i] != q.shape[i] || !small(q.shape[i])) return closer();
    if (q.shape[2] != p.dim || tables.dtype != at::kInt || tables.dims != 2 || tables.shape[0] != q.shape[0] ||
        !small(tables.shape[1]) || tables.device != dev || !is_vector(&lens, at::kInt, q.shape[0], dev))
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
PyObject* prefill_window(PyObject* const* a, Py_ssize_t n) {
    Pools p;
    Info out, q, tables, start, cu;
    int32_t chunk, window, sinks, *err;
    void* raw;
    if (n != 13 || look_pools(a[2], a[3], PA_BF16, &p) < 0) return closer();
    const long dev = p.k.device;
    if (look(a[0], &out, false) < 0 || look(a[1], &q, false) < 0 || look(a[4], &tables, false) < 0 || look(a[5], &start, false) < 0 ||
        look(a[6], &cu, false) < 0)
        return closer();
    if (q.dtype != p.rows || out.dtype != p.rows || q.dims != 3 || out.dims != 3 || q.device != dev || out.device != dev)
        return closer();
    for (int i = 0; i < 3; ++i)
        if (out.shape[i] != q.shape[i] || !small(q.shape[i])) return closer();
    if (q.shape[2] != p.dim || tables.dtype != at::kInt || tables.dims != 2 || !small(tables.shape[0]) ||
        !small(tables.shape[1]) || tables.device != dev || !is_vector(&start, at::kInt, tables.shape[0], dev) ||
        !is_vector(&cu, at::kInt, tables.shape[0] + 1, dev))
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
int look_rows(PyObject* t, const Pools* p, int64_t n, int64_t heads, Info* x) {
    if (look(t, x, true) < 0 || x->dtype != p->rows || x->dims != 3 || x->device != p->k.device) return -1;
    if ((n >= 0 && x->shape[0] != n) || (heads >= 0 && x->shape[1] != heads) || x->shape[2] != p->dim) return -1;
    if (!small(x->shape[0]) || !small(x->shape[1])) return -1;
    if (x->stride[2] != 1 || x->stride[1] != p->dim) return -1;
    if (x->shape[0] <= 1) x->stride[0] = x->shape[1] * p->dim;
    return 0;
}

/* rope_append(kind, k_pool, v_pool, q_out, q, k_new, v_new, inv_freq, tables, start, cu, interleaved, flag, stream) */
PyObject* rope_append(PyObject* const* a, Py_ssize_t n) {
    Pools p;
    Info qo, q, k, v, freq, tables, start, cu;
    int32_t* err;
    void* raw;
    if (n != 14 || look_pools(a[1], a[2], PyLong_AsLong(a[0]), &p) < 0) return closer();
    const long dev = p.k.device;
    if (look_rows(a[5], &p, -1, p.heads, &k) < 0 || look_rows(a[6], &p, k.shape[0], p.heads, &v) < 0) return closer();
    if (a[4] == Py_None && a[3] == Py_None) {
        q.ptr.at = qo.ptr.at = nullptr;
        q.shape[1] = q.stride[0] = qo.stride[0] = 0;
    } else if (look_rows(a[4], &p, k.shape[0], -1, &q) < 0 || look_rows(a[3], &p, k.shape[0], q.shape[1], &qo) < 0) {
        return closer();
    }
    if (look(a[7], &freq, false) < 0 || look(a[8], &tables, false) < 0 || look(a[9], &start, false) < 0 || look(a[10], &cu, false) < 0)
        return closer();
    if (freq.dims != 1 || freq.shape[0] > 1 << 20 || !is_vector(&freq, at::kDouble, freq.shape[0], dev) || tables.dtype != at::kInt ||
        tables.dims != 2 || !small(tables.shape[0]) || !small(tables.shape[1]) || tables.device != dev ||
        !is_vector(&start, at::kInt, tables.shape[0], dev) || !is_vector(&cu, at::kInt, tables.shape[0] + 1, dev))
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

/* A call, with -1 where torch throws (a tensor without memory, for instance). */
template <PyObject* (*Call)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!call_rope) return closer();
    try {
        return Call(a, n);
    } catch (...) {
        return closer();
    }
}

/* bind(rope, decode, prefill): the addresses of the library's functions, once, before any other call. */
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void* at[3];
    if (n != 3) {
        PyErr_SetString(PyExc_TypeError, "bind: three addresses");
        return nullptr;
    }
    for (int i = 0; i < 3; ++i) {
        at[i] = PyLong_AsVoidPtr(a[i]);
        if (!at[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null address");
            return nullptr;
        }
    }
    call_decode = reinterpret_cast<decode_fn>(at[1]);
    call_prefill = reinterpret_cast<prefill_fn>(at[2]);
    call_rope = reinterpret_cast<rope_fn>(at[0]);
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f));
}
PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"rope_append", fast(guarded<rope_append>), METH_FASTCALL, nullptr},
                         {"decode_window", fast(guarded<decode_window>), METH_FASTCALL, nullptr},
                         {"prefill_window", fast(guarded<prefill_window>), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_quick", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__quick(void) {
    PyObject* m = PyModule_Create(&module);
    /* tensors are read as this version of torch lays them out */
    if (m && PyModule_AddStringConstant(m, "torch_version", PA_TORCH_VERSION) < 0) Py_CLEAR(m);
    return m;
}
