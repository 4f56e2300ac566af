// Native argument marshalling of the attention sublayer's Python functions.
//
// A decode step calls them eagerly with a dozen small tensors, and checking
// those in Python takes longer than the kernels run (norm and rotation of 8
// tokens: 8.1 us a call, of which 4 are the checks and 3.3 the launch).  Each
// function here reads its tensors through DLPack's exchange interface, checks
// what the Python function checks, and calls the C entry point on the
// device's current stream.  It returns True when that call returned BEAM_OK
// (3.7 us for the call above).
// Whatever does not fit, here or in the entry point's own checks, returns
// False with nothing enqueued, and the Python function then goes its own way,
// which names what is wrong.  A call that failed in HIP may have enqueued work
// (in place, it must not be made twice): it raises.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/dlpack.h>
#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "beam_moe.h"

namespace {

const DLPackExchangeAPI* g_api = nullptr;
int g_gpu_type = 0;   // DLPack's device type of this torch's GPU tensors
PyObject* g_error = nullptr;   // what a failed call raises: g_error(entry point, status)

decltype(&beam_moe_qk_norm_rope) g_norm_rope = nullptr;
decltype(&beam_moe_qk_norm_rope_cache) g_norm_rope_cache = nullptr;
decltype(&beam_moe_kv_write) g_kv_write = nullptr;
decltype(&beam_moe_kv_read) g_kv_read = nullptr;
decltype(&beam_moe_attn_decode) g_decode = nullptr;

constexpr DLDataType kF32{kDLFloat, 32, 1}, kBF16{kDLBfloat, 16, 1}, kI32{kDLInt, 32, 1}, kU8{kDLUInt, 8, 1};

bool same(DLDataType a, DLDataType b) { return a.code == b.code && a.bits == b.bits && a.lanes == b.lanes; }

bool view(PyObject* o, DLTensor& t) {
    if (g_api->dltensor_from_py_object_no_sync(o, &t) == 0) return true;
    PyErr_Clear();
    return false;
}

void* data(const DLTensor& t) { return static_cast<char*>(t.data) + t.byte_offset; }

// shape, dtype and device of a tensor; *out its data
bool fits(const DLTensor& t, int dev, DLDataType dt, int nd, const int64_t* shape) {
    if ((int)t.device.device_type != g_gpu_type || t.device.device_id != dev || !same(t.dtype, dt) || t.ndim != nd)
        return false;
    for (int i = 0; i < nd; ++i)
        if (t.shape[i] != shape[i]) return false;
    return true;
}
bool contiguous(const DLTensor& t) {
    if (!t.strides) return true;
    int64_t want = 1;
    for (int i = t.ndim - 1; i >= 0; --i) {
        if (t.shape[i] != 1 && t.strides[i] != want) return false;
        want *= t.shape[i];
    }
    return true;
}
bool dense(PyObject* o, int dev, DLDataType dt, int nd, const int64_t* shape, void** out) {
    DLTensor t;
    if (!view(o, t) || !fits(t, dev, dt, nd, shape) || !contiguous(t)) return false;
    *out = data(t);
    return true;
}
bool dense1(PyObject* o, int dev, DLDataType dt, int64_t n, void** out) { return dense(o, dev, dt, 1, &n, out); }
bool dense1_or_none(PyObject* o, int dev, DLDataType dt, int64_t n, void** out) {
    *out = nullptr;
    return o == Py_None || dense1(o, dev, dt, n, out);
}

// [T, heads, dim] rows whose heads are adjacent
bool heads(const DLTensor& t, int dev, DLDataType dt, int64_t T, int64_t n, int64_t dim, void** out, int64_t* stride) {
    const int64_t shape[3] = {T, n, dim};
    if (!fits(t, dev, dt, 3, shape)) return false;
    if (t.strides && (t.strides[2] != 1 || (t.strides[1] != dim && n > 1))) return false;
    *out = data(t);
    *stride = t.strides && T > 1 ? t.strides[0] : n * dim;
    return true;
}
bool heads(PyObject* o, int dev, DLDataType dt, int64_t T, int64_t n, int64_t dim, void** out, int64_t* stride) {
    DLTensor t;
    return view(o, t) && heads(t, dev, dt, T, n, dim, out, stride);
}

// The C struct inside a ctypes structure object (alive as long as the caller's
// argument is).
template <typename S> const S* struct_of(PyObject* o) {
    Py_buffer b;
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) {
        PyErr_Clear();
        return nullptr;
    }
    const S* p = b.len == (Py_ssize_t)sizeof(S) ? static_cast<const S*>(b.buf) : nullptr;
    PyBuffer_Release(&b);
    return p;
}

// What the calls have in common: the device and its current stream, rows and
// dtype of the activations, the shape of the layer.
struct Call {
    const beam_moe_attn_cfg* cfg;
    int dev;
    int64_t T;
    DLDataType dt;
    beam_dtype code;
    void* stream;
};
bool open_call(PyObject* cfg, const DLTensor& act, Call& c) {
    c.cfg = struct_of<beam_moe_attn_cfg>(cfg);
    if (!c.cfg) return false;
    c.dev = act.device.device_id;
    if ((int)act.device.device_type != g_gpu_type || act.ndim != 3) return false;
    c.T = act.shape[0];
    c.dt = act.dtype;
    if (same(c.dt, kBF16)) c.code = BEAM_BF16;
    else if (same(c.dt, kF32)) c.code = BEAM_F32;
    else return false;
    if (c.T > INT32_MAX) return false;
    c.stream = nullptr;
    if (g_gpu_type == kDLCPU) return true;   // bound for host tensors: no current device, no stream
    int cur = -1;
    if (hipGetDevice(&cur) != hipSuccess || cur != c.dev) return false;
    if (g_api->current_work_stream(act.device.device_type, c.dev, &c.stream) != 0) {
        PyErr_Clear();
        return false;
    }
    return true;
}

// The cache struct that a KVCache made, if its keys still are where they were
// and have the layer's page shape.
const beam_moe_kv_cache* cache_of(const Call& c, PyObject* cache, PyObject* k) {
    const auto* kv = struct_of<beam_moe_kv_cache>(cache);
    DLTensor t;
    if (!kv || !view(k, t)) return nullptr;
    if ((int)t.device.device_type != g_gpu_type || t.device.device_id != c.dev || t.ndim != 4 || data(t) != kv->k ||
        t.shape[0] != kv->n_pages || t.shape[1] != c.cfg->n_kv_heads || t.shape[2] != c.cfg->page_size ||
        t.shape[3] != c.cfg->head_dim)
        return nullptr;
    return kv;
}

PyObject* does_not_fit() { Py_RETURN_FALSE; }

// What a made call comes to.
PyObject* outcome(const char* fn, beam_status st) {
    if (st == BEAM_OK) Py_RETURN_TRUE;
    if (st == BEAM_ERR_INVALID_ARG || st == BEAM_ERR_UNSUPPORTED || st == BEAM_ERR_WORKSPACE) Py_RETURN_FALSE;
    PyObject* e = PyObject_CallFunction(g_error, "si", fn, (int)st);
    if (e) PyErr_SetObject(g_error, e);
    Py_XDECREF(e);
    return nullptr;
}

struct Prep {
    void *q, *k, *gq, *gk, *pos, *freq, *q_out;
    int64_t qs, ks;
};
// q, k, positions, q_out, inv_freq, gamma_q, gamma_k
bool prep(Call& c, PyObject* cfg, PyObject* q, PyObject* k, PyObject* pos, PyObject* q_out, PyObject* freq,
          PyObject* gq, PyObject* gk, Prep& p) {
    DLTensor t;
    if (!view(q, t) || !open_call(cfg, t, c)) return false;
    const int64_t D = c.cfg->head_dim, qshape[3] = {c.T, c.cfg->n_heads, D};
    if (!heads(t, c.dev, c.dt, c.T, c.cfg->n_heads, D, &p.q, &p.qs)) return false;
    if (!heads(k, c.dev, c.dt, c.T, c.cfg->n_kv_heads, D, &p.k, &p.ks)) return false;
    if (!dense1(pos, c.dev, kI32, c.T, &p.pos) || !dense(q_out, c.dev, c.dt, 3, qshape, &p.q_out)) return false;
    p.freq = nullptr;
    if (c.cfg->rope_dim && !dense1(freq, c.dev, kF32, c.cfg->rope_dim / 2, &p.freq)) return false;
    return dense1_or_none(gq, c.dev, c.dt, D, &p.gq) && dense1_or_none(gk, c.dev, c.dt, D, &p.gk);
}

// (cfg, q, k, positions, q_out, k_out, inv_freq, gamma_q, gamma_k)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    Call c;
    Prep p;
    void* k_out;
    if (n != 9 || !g_norm_rope || !prep(c, a[0], a[1], a[2], a[3], a[4], a[6], a[7], a[8], p)) return does_not_fit();
    const int64_t ks[3] = {c.T, c.cfg->n_kv_heads, c.cfg->head_dim};
    if (!dense(a[5], c.dev, c.dt, 3, ks, &k_out)) return does_not_fit();
    const beam_status st = g_norm_rope(c.cfg, (int32_t)c.T, p.q, p.qs, p.k, p.ks, c.code, p.gq, p.gk,
                                       static_cast<const int32_t*>(p.pos), static_cast<const float*>(p.freq), p.q_out,
                                       k_out, c.stream);
    return outcome("beam_moe_qk_norm_rope", st);
}

// (cfg, q, k, v, positions, slots, q_out, cache, cache.k, inv_freq, gamma_q, gamma_k)
PyObject* qk_norm_rope_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
    Call c;
    Prep p;
    void *v, *slots;
    int64_t vs;
    if (n != 12 || !g_norm_rope_cache || !prep(c, a[0], a[1], a[2], a[4], a[6], a[9], a[10], a[11], p))
        return does_not_fit();
    const beam_moe_kv_cache* kv = cache_of(c, a[7], a[8]);
    if (!kv || !heads(a[3], c.dev, c.dt, c.T, c.cfg->n_kv_heads, c.cfg->head_dim, &v, &vs) ||
        !dense1(a[5], c.dev, kI32, c.T, &slots))
        return does_not_fit();
    const beam_status st = g_norm_rope_cache(c.cfg, (int32_t)c.T, p.q, p.qs, p.k, p.ks, v, vs, c.code, p.gq, p.gk,
                                             static_cast<const int32_t*>(p.pos), static_cast<const float*>(p.freq),
                                             static_cast<const int32_t*>(slots), p.q_out, kv, c.stream);
    return outcome("beam_moe_qk_norm_rope_cache", st);
}

// (cfg, k, v, slots, cache, cache.k)
PyObject* kv_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
    Call c;
    DLTensor t;
    void *k, *v, *slots;
    int64_t ks, vs;
    if (n != 6 || !g_kv_write || !view(a[1], t) || !open_call(a[0], t, c)) return does_not_fit();
    const int64_t h = c.cfg->n_kv_heads, D = c.cfg->head_dim;
    const beam_moe_kv_cache* kv = cache_of(c, a[4], a[5]);
    if (!kv || !heads(t, c.dev, c.dt, c.T, h, D, &k, &ks) || !heads(a[2], c.dev, c.dt, c.T, h, D, &v, &vs) ||
        !dense1(a[3], c.dev, kI32, c.T, &slots))
        return does_not_fit();
    const beam_status st = g_kv_write(c.cfg, (int32_t)c.T, k, ks, v, vs, c.code, static_cast<const int32_t*>(slots), kv,
                                      c.stream);
    return outcome("beam_moe_kv_write", st);
}

// [B, width] int32 page table; B and width come out
bool page_table(PyObject* o, int dev, int64_t* B, int64_t* width, void** out) {
    DLTensor t;
    if (!view(o, t) || t.ndim != 2 || !contiguous(t)) return false;
    if (*B < 0) *B = t.shape[0];
    const int64_t shape[2] = {*B, t.shape[1]};
    *width = t.shape[1];
    *out = data(t);
    return fits(t, dev, kI32, 2, shape) && *B <= INT32_MAX && *width <= INT32_MAX;
}

// (cfg, cache, cache.k, page_table, row_offsets, k_out, v_out, first)
PyObject* kv_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    Call c;
    DLTensor t;
    void *table, *off, *k, *v, *first;
    int64_t B = -1, width;
    if (n != 8 || !g_kv_read || !view(a[5], t) || !open_call(a[0], t, c)) return does_not_fit();
    const int64_t shape[3] = {c.T, c.cfg->n_kv_heads, c.cfg->head_dim};
    const beam_moe_kv_cache* kv = cache_of(c, a[1], a[2]);
    if (!kv || !fits(t, c.dev, c.dt, 3, shape) || !contiguous(t) || !dense(a[6], c.dev, c.dt, 3, shape, &v) ||
        !page_table(a[3], c.dev, &B, &width, &table) || !dense1(a[4], c.dev, kI32, B + 1, &off) ||
        !dense1_or_none(a[7], c.dev, kI32, B, &first))
        return does_not_fit();
    k = data(t);
    const beam_status st = g_kv_read(c.cfg, (int32_t)B, (int32_t)c.T, kv, static_cast<const int32_t*>(table),
                                     (int32_t)width, static_cast<const int32_t*>(off),
                                     static_cast<const int32_t*>(first), k, v, c.code, c.stream);
    return outcome("beam_moe_kv_read", st);
}

// (cfg, q, cache, cache.k, page_table, seq_lens, max_len, out, ws, lse)
PyObject* attn_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    Call c;
    DLTensor t, w;
    void *q, *table, *lens, *out, *lse = nullptr, *ws = nullptr;
    int64_t qs, width, wn = 0;
    if (n != 10 || !g_decode || !view(a[1], t) || !open_call(a[0], t, c)) return does_not_fit();
    const int64_t h = c.cfg->n_heads, D = c.cfg->head_dim, shape[3] = {c.T, h, D}, ls[2] = {c.T, h};
    int64_t B = c.T;
    const beam_moe_kv_cache* kv = cache_of(c, a[2], a[3]);
    const long long max_len = PyLong_AsLongLong(a[6]);
    if (max_len == -1 && PyErr_Occurred()) PyErr_Clear();
    if (!kv || max_len < 0 || max_len > INT32_MAX || !heads(t, c.dev, c.dt, B, h, D, &q, &qs) ||
        !page_table(a[4], c.dev, &B, &width, &table) || !dense1(a[5], c.dev, kI32, B, &lens) ||
        !dense(a[7], c.dev, c.dt, 3, shape, &out))
        return does_not_fit();
    if (a[9] != Py_None && !dense(a[9], c.dev, kF32, 2, ls, &lse)) return does_not_fit();
    if (a[8] != Py_None) {
        if (!view(a[8], w) || w.ndim != 1 || !fits(w, c.dev, kU8, 1, w.shape) || !contiguous(w)) return does_not_fit();
        ws = data(w);
        wn = w.shape[0];
    }
    const beam_status st = g_decode(c.cfg, (int32_t)B, q, qs, c.code, kv, static_cast<const int32_t*>(table),
                                    (int32_t)width, static_cast<const int32_t*>(lens), (int32_t)max_len, out,
                                    static_cast<float*>(lse), ws, (size_t)wn, c.stream);
    return outcome("beam_moe_attn_decode", st);
}

// bind(exchange capsule, gpu device type, addresses of the five entry points[,
// class of the errors])
PyObject* bind(PyObject*, PyObject* args) {
    PyObject *cap, *error = PyExc_RuntimeError;
    int type;
    unsigned long long f[5];
    if (!PyArg_ParseTuple(args, "OiKKKKK|O", &cap, &type, &f[0], &f[1], &f[2], &f[3], &f[4], &error)) return nullptr;
    if (!PyExceptionClass_Check(error)) {
        PyErr_SetString(PyExc_TypeError, "not an exception class");
        return nullptr;
    }
    auto* api = static_cast<const DLPackExchangeAPI*>(PyCapsule_GetPointer(cap, "dlpack_exchange_api"));
    if (!api) return nullptr;
    if (api->header.version.major != DLPACK_MAJOR_VERSION || !api->dltensor_from_py_object_no_sync ||
        !api->current_work_stream) {
        PyErr_SetString(PyExc_RuntimeError, "this torch's DLPack exchange interface is not the one built for");
        return nullptr;
    }
    g_api = api;
    g_gpu_type = type;
    Py_INCREF(error);
    Py_XDECREF(g_error);
    g_error = error;
    g_norm_rope = reinterpret_cast<decltype(g_norm_rope)>(f[0]);
    g_norm_rope_cache = reinterpret_cast<decltype(g_norm_rope_cache)>(f[1]);
    g_kv_write = reinterpret_cast<decltype(g_kv_write)>(f[2]);
    g_kv_read = reinterpret_cast<decltype(g_kv_read)>(f[3]);
    g_decode = reinterpret_cast<decltype(g_decode)>(f[4]);
    Py_RETURN_NONE;
}

template <typename F> PyMethodDef fast(const char* name, F f) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {fast("qk_norm_rope", qk_norm_rope),
                         fast("qk_norm_rope_cache", qk_norm_rope_cache),
                         fast("kv_write", kv_write),
                         fast("kv_read", kv_read),
                         fast("attn_decode", attn_decode),
                         {"bind", bind, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
