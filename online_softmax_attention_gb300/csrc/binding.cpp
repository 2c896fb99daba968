// Calls of the library straight from torch tensors, for short calls.
//
// The Python binding checks and packs its arguments in the interpreter, which
// costs more than a short attention takes on the GPU (decoding one sequence: 25
// us of host time around 11 us of kernels).  The functions here do the same for
// arguments that need no conversion -- CUDA tensors of one device, which is
// current, of the expected types and shapes, lists already int32 vectors there --
// and return None for anything else: the Python path then converts the arguments
// or names what is wrong with them.  A status other than 0 is returned as a
// number, which the caller turns into the exception.
//
// Every step of the computation runs in the CUDA library; this file marshals.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>

#include "../../include/attn.h"

namespace {

using at::Tensor;

struct Api {
    decltype(&attn_fwd) fwd;
    decltype(&attn_fwd_workspace_bytes) fwd_bytes;
    decltype(&attn_bwd) bwd;
    decltype(&attn_bwd_workspace_bytes) bwd_bytes;
    decltype(&attn_tree_fwd) tree;
    decltype(&attn_tree_workspace_bytes) tree_bytes;
    decltype(&attn_cache_workspace_bytes) cache_bytes;
    decltype(&attn_cache_extend) extend;
    decltype(&attn_cache_fork) fork;
    decltype(&attn_cache_keep) keep;
    decltype(&attn_cache_free) free;
    decltype(&attn_cache_write) write;
    decltype(&attn_cache_weigh) weigh;
    decltype(&attn_weigh_workspace_bytes) weigh_bytes;
    decltype(&attn_cache_evict) evict;
    decltype(&attn_cache_evict_workspace_bytes) evict_bytes;
} api;

// A call's conditions: the first that does not hold ends it with None.
#define NEED(cond) \
    if (!(cond)) Py_RETURN_NONE

const Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

int dtype_code(const Tensor &t) {
    switch (t.scalar_type()) {
    case at::kHalf: return ATTN_F16;
    case at::kBFloat16: return ATTN_BF16;
    case at::kFloat: return ATTN_F32;
    default: return -1;
    }
}

at::ScalarType scalar_of(int code) {
    return code == ATTN_F16 ? at::kHalf : code == ATTN_BF16 ? at::kBFloat16 : at::kFloat;
}

// The device of a call: the tensor's, if it is current.  -1: not a plain case.
int device_of(const Tensor *t) {
    if (!t || !t->is_cuda()) return -1;
    const int d = t->get_device();
    return d == c10::cuda::current_device() ? d : -1;
}

bool on(const Tensor *t, int device) { return t && t->is_cuda() && t->get_device() == device; }

// A (tokens, heads, D) tensor with contiguous D.
bool rows(const Tensor *t, int device, int64_t D, attn_tensor &v) {
    if (!on(t, device) || t->dim() != 3 || t->size(2) != D || t->stride(2) != 1) return false;
    // a size-1 axis is never stepped along, so any aligned stride describes it
    v.ptr = t->size(0) ? t->data_ptr() : nullptr;
    v.stride_tok = t->size(0) > 1 ? t->stride(0) : t->size(1) * D;
    v.stride_head = t->size(1) > 1 ? t->stride(1) : D;
    return true;
}

// An int32 vector.
bool ints(const Tensor *t, int device) {
    return on(t, device) && t->dim() == 1 && t->scalar_type() == at::kInt && t->is_contiguous();
}

const int32_t *int_ptr(const Tensor *t) { return static_cast<const int32_t *>(t->data_ptr()); }

Tensor empty(at::IntArrayRef size, at::ScalarType type, int device) {
    return at::empty(size, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, device)));
}

Tensor scratch(size_t bytes, int device) { return empty({(int64_t)(bytes > 256 ? bytes : 256)}, at::kByte, device); }

void *stream_of(int device) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }

PyObject *status(int rc) { return PyLong_FromLong(rc); }

PyObject *pack(std::initializer_list<Tensor> ts) {
    PyObject *r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) return nullptr;
    Py_ssize_t i = 0;
    for (const Tensor &t : ts) {
        PyObject *o = THPVariable_Wrap(t);
        if (!o) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

bool as_long(PyObject *o, long &v) {
    if (!PyLong_Check(o)) return false;
    v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    return v >= INT32_MIN && v <= INT32_MAX;
}

// A float in a C float's range, or None for D^-1/2.
bool as_scale(PyObject *o, int64_t D, float &v) {
    if (o == Py_None) {
        v = (float)(1.0 / std::sqrt((double)D));
        return true;
    }
    if (!PyFloat_Check(o)) return false;
    const double x = PyFloat_AS_DOUBLE(o);
    v = (float)x;
    return std::isfinite(x) && std::isfinite(v);
}

bool fits(int64_t n) { return n <= INT32_MAX; }

// A sliding window's arguments: None and 0, or window >= 1 and sinks >= 0.
bool windowed(PyObject *window, PyObject *sinks, int32_t &w, int32_t &s) {
    long x = 0, y = 0;
    if (PyBool_Check(window) || PyBool_Check(sinks) || !as_long(sinks, y) || y < 0) return false;
    if (window == Py_None ? y != 0 : !as_long(window, x) || x < 1) return false;
    w = (int32_t)x;
    s = (int32_t)y;
    return true;
}

// The device lists of offsets of a call: none, or int32 vectors.
bool offsets(PyObject *oq, PyObject *ok, int device, const int32_t *&cq, const int32_t *&ck, int32_t &n_seq) {
    cq = ck = nullptr;
    n_seq = 1;
    if (oq == Py_None) return ok == Py_None;
    const Tensor *tq = tensor(oq), *tk = ok == Py_None ? tq : tensor(ok);
    if (!ints(tq, device) || !ints(tk, device) || tq->size(0) < 2 || tk->size(0) != tq->size(0)) return false;
    cq = int_ptr(tq);
    ck = int_ptr(tk);
    n_seq = (int32_t)(tq->size(0) - 1);
    return true;
}

// fwd(q, k, v, causal, scale, cu_q, cu_k, out_code, window, sinks) -> (o, lse) | status | None
PyObject *py_fwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    NEED(n == 10);
    const Tensor *q = tensor(args[0]), *k = tensor(args[1]), *v = tensor(args[2]);
    const int dev = device_of(q);
    NEED(dev >= 0 && k && v && q->dim() == 3 && k->dim() == 3 && v->dim() == 3);
    const int64_t T = q->size(0), H = q->size(1), D = q->size(2);
    attn_fwd_args a;
    std::memset(&a, 0, sizeof(a));
    NEED(windowed(args[8], args[9], a.window, a.sinks));
    NEED(rows(q, dev, D, a.q) && rows(k, dev, D, a.k) && rows(v, dev, D, a.v));
    const int code = dtype_code(*q);
    NEED(code >= 0 && dtype_code(*k) == code && dtype_code(*v) == code && k->sizes() == v->sizes());
    long out;
    NEED(as_long(args[7], out) && T > 0 && k->size(0) > 0 && k->size(1) > 0 && fits(T * H) && fits(k->size(0)));
    if (out < 0) out = code;
    NEED((out == code || out == ATTN_F32) && as_scale(args[4], D, a.scale));
    NEED(offsets(args[5], args[6], dev, a.cu_seqlens_q, a.cu_seqlens_k, a.n_seq));
    a.n_q = (int32_t)T;
    a.n_k = (int32_t)k->size(0);
    a.H = (int32_t)H;
    a.D = (int32_t)D;
    a.H_kv = (int32_t)k->size(1);
    a.relation = args[3] == Py_True ? ATTN_CAUSAL : ATTN_FULL;
    NEED(args[3] == Py_True || args[3] == Py_False);
    a.dtype = code;
    a.o_dtype = (int32_t)out;
    Tensor o = empty(q->sizes(), scalar_of((int)out), dev), lse = empty({H, T}, at::kFloat, dev);
    a.o.ptr = o.data_ptr();
    a.o.stride_tok = H * D;
    a.o.stride_head = D;
    a.lse = static_cast<float *>(lse.data_ptr());
    const Tensor ws = scratch(api.fwd_bytes(&a), dev);
    a.workspace = ws.data_ptr();
    a.workspace_bytes = (size_t)ws.size(0);
    const int rc = api.fwd(&a, stream_of(dev));
    return rc ? status(rc) : pack({o, lse});
}

// bwd(q, k, v, o, lse, dout, causal, scale, cu_q, cu_k, grad_code, window, sinks) -> (dq, dk, dv) | status | None
PyObject *py_bwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    NEED(n == 13);
    const Tensor *q = tensor(args[0]), *k = tensor(args[1]), *v = tensor(args[2]), *o = tensor(args[3]),
                 *lse = tensor(args[4]), *d = tensor(args[5]);
    const int dev = device_of(q);
    NEED(dev >= 0 && k && v && o && lse && d && q->dim() == 3 && k->dim() == 3);
    const int64_t T = q->size(0), H = q->size(1), D = q->size(2);
    attn_bwd_args a;
    std::memset(&a, 0, sizeof(a));
    NEED(windowed(args[11], args[12], a.window, a.sinks));
    NEED(rows(q, dev, D, a.q) && rows(k, dev, D, a.k) && rows(v, dev, D, a.v) && rows(o, dev, D, a.o) &&
         rows(d, dev, D, a.dout));
    const int code = dtype_code(*q), o_code = dtype_code(*o);
    NEED(code >= 0 && dtype_code(*k) == code && dtype_code(*v) == code && dtype_code(*d) == code &&
         (o_code == code || o_code == ATTN_F32) && k->sizes() == v->sizes() && o->sizes() == q->sizes() &&
         d->sizes() == q->sizes());
    NEED(on(lse, dev) && lse->scalar_type() == at::kFloat && lse->dim() == 2 && lse->size(0) == H &&
         lse->size(1) == T && lse->is_contiguous());
    long grad;
    NEED(as_long(args[10], grad) && T > 0 && k->size(0) > 0 && k->size(1) > 0 && fits(T * H) && fits(k->size(0)));
    if (grad < 0) grad = code;
    NEED((grad == code || grad == ATTN_F32) && as_scale(args[7], D, a.scale));
    NEED(args[6] == Py_True || args[6] == Py_False);
    NEED(offsets(args[8], args[9], dev, a.cu_seqlens_q, a.cu_seqlens_k, a.n_seq));
    const int64_t Hk = k->size(1);
    a.lse = static_cast<const float *>(lse->data_ptr());
    a.n_q = (int32_t)T;
    a.n_k = (int32_t)k->size(0);
    a.H = (int32_t)H;
    a.D = (int32_t)D;
    a.H_kv = (int32_t)Hk;
    a.relation = args[6] == Py_True ? ATTN_CAUSAL : ATTN_FULL;
    a.dtype = code;
    a.o_dtype = o_code;
    a.grad_dtype = (int32_t)grad;
    const at::ScalarType type = scalar_of((int)grad);
    Tensor dq = empty(q->sizes(), type, dev), dk = empty(k->sizes(), type, dev), dv = empty(k->sizes(), type, dev);
    a.dq = attn_tensor{dq.data_ptr(), H * D, D};
    a.dk = attn_tensor{dk.data_ptr(), Hk * D, D};
    a.dv = attn_tensor{dv.data_ptr(), Hk * D, D};
    const Tensor ws = scratch(api.bwd_bytes(&a), dev);
    a.workspace = ws.data_ptr();
    a.workspace_bytes = (size_t)ws.size(0);
    const int rc = api.bwd(&a, stream_of(dev));
    return rc ? status(rc) : pack({dq, dk, dv});
}

// The cache behind a call: its packed description and its device.
bool cache_of(PyObject *bytes, PyObject *index, attn_cache &c, int &dev) {
    long d;
    if (!PyBytes_Check(bytes) || PyBytes_GET_SIZE(bytes) != (Py_ssize_t)sizeof(c) || !as_long(index, d)) return false;
    std::memcpy(&c, PyBytes_AS_STRING(bytes), sizeof(c));
    dev = (int)d;
    return dev == c10::cuda::current_device();
}

// tree(cache, device, q, seqs, cu, mask, layer, scale, out_code, window, sinks) -> (o, lse) | status | None
PyObject *py_tree(PyObject *, PyObject *const *args, Py_ssize_t n) {
    attn_tree_args a;
    std::memset(&a, 0, sizeof(a));
    int dev;
    NEED(n == 11 && cache_of(args[0], args[1], a.cache, dev) && windowed(args[9], args[10], a.window, a.sinks));
    const Tensor *q = tensor(args[2]), *seqs = tensor(args[3]), *cu = tensor(args[4]);
    long layer, out;
    NEED(q && rows(q, dev, a.cache.D, a.q) && dtype_code(*q) == a.cache.dtype && ints(seqs, dev) && ints(cu, dev));
    NEED(cu->size(0) == seqs->size(0) + 1 && as_long(args[6], layer) && as_long(args[8], out));
    const int64_t T = q->size(0), H = q->size(1), D = a.cache.D;
    if (out < 0) out = a.cache.dtype;
    NEED((out == a.cache.dtype || out == ATTN_F32) && as_scale(args[7], D, a.scale) && T > 0 && fits(T * H) &&
         fits(seqs->size(0)));
    if (args[5] != Py_None) {
        const Tensor *m = tensor(args[5]);
        NEED(on(m, dev) && m->scalar_type() == at::kLong && m->dim() == 2 && m->size(0) == T && m->size(1) >= 1 &&
             fits(m->size(1)) && m->is_contiguous());
        a.mask = static_cast<const uint64_t *>(m->data_ptr());
        a.mask_words = (int32_t)m->size(1);
    }
    Tensor o = empty(q->sizes(), scalar_of((int)out), dev), lse = empty({H, T}, at::kFloat, dev);
    a.layer = (int32_t)layer;
    a.H = (int32_t)H;
    a.o = attn_tensor{o.data_ptr(), H * D, D};
    a.lse = static_cast<float *>(lse.data_ptr());
    a.seqs = int_ptr(seqs);
    a.cu = int_ptr(cu);
    a.n = (int32_t)seqs->size(0);
    a.n_q = (int32_t)T;
    a.o_dtype = (int32_t)out;
    const Tensor ws = scratch(api.tree_bytes(&a), dev);
    a.workspace = ws.data_ptr();
    a.workspace_bytes = (size_t)ws.size(0);
    const int rc = api.tree(&a, stream_of(dev));
    return rc ? status(rc) : pack({o, lse});
}

// write(cache, device, seqs, cu, k, v, layer) -> status | None
PyObject *py_write(PyObject *, PyObject *const *args, Py_ssize_t n) {
    attn_cache c;
    int dev;
    NEED(n == 7 && cache_of(args[0], args[1], c, dev));
    const Tensor *seqs = tensor(args[2]), *cu = tensor(args[3]), *k = tensor(args[4]), *v = tensor(args[5]);
    attn_tensor kt, vt;
    long layer;
    NEED(ints(seqs, dev) && ints(cu, dev) && cu->size(0) == seqs->size(0) + 1 && k && v && rows(k, dev, c.D, kt) &&
         rows(v, dev, c.D, vt) && as_long(args[6], layer));
    NEED(k->sizes() == v->sizes() && k->size(1) == c.H_kv && dtype_code(*k) == c.dtype && dtype_code(*v) == c.dtype &&
         fits(k->size(0)) && fits(seqs->size(0)));
    return status(api.write(&c, (int32_t)layer, int_ptr(seqs), int_ptr(cu), (int32_t)seqs->size(0), &kt, &vt,
                            (int32_t)k->size(0), stream_of(dev)));
}

// extend / fork(cache, device, a, b) -> status | None
template <bool kFork>
PyObject *py_alloc(PyObject *, PyObject *const *args, Py_ssize_t n) {
    attn_cache c;
    int dev;
    NEED(n == 4 && cache_of(args[0], args[1], c, dev));
    const Tensor *x = tensor(args[2]), *y = tensor(args[3]);
    NEED(ints(x, dev) && ints(y, dev) && x->size(0) == y->size(0) && fits(x->size(0)));
    const Tensor ws = scratch(api.cache_bytes(&c, (int32_t)x->size(0)), dev);
    return status((kFork ? api.fork : api.extend)(&c, int_ptr(x), int_ptr(y), (int32_t)x->size(0), ws.data_ptr(),
                                                  (size_t)ws.size(0), stream_of(dev)));
}

// keep(cache, device, seqs, n_draft, keep, n_keep) -> status | None
PyObject *py_keep(PyObject *, PyObject *const *args, Py_ssize_t n) {
    attn_cache c;
    int dev;
    NEED(n == 6 && cache_of(args[0], args[1], c, dev));
    const Tensor *s = tensor(args[2]), *d = tensor(args[3]), *k = tensor(args[4]), *m = tensor(args[5]);
    NEED(ints(s, dev) && ints(d, dev) && ints(m, dev) && on(k, dev) && k->dim() == 2 &&
         k->scalar_type() == at::kInt && k->is_contiguous() && fits(s->size(0)));
    NEED(d->size(0) == s->size(0) && m->size(0) == s->size(0) && k->size(0) == s->size(0));
    const Tensor ws = scratch(api.cache_bytes(&c, (int32_t)s->size(0)), dev);
    return status(api.keep(&c, int_ptr(s), int_ptr(d), int_ptr(k), k->size(1), int_ptr(m), (int32_t)s->size(0),
                           ws.data_ptr(), (size_t)ws.size(0), stream_of(dev)));
}

// free(cache, device, seqs) -> status | None
PyObject *py_free(PyObject *, PyObject *const *args, Py_ssize_t n) {
    attn_cache c;
    int dev;
    NEED(n == 3 && cache_of(args[0], args[1], c, dev));
    const Tensor *s = tensor(args[2]);
    NEED(ints(s, dev) && fits(s->size(0)));
    return status(api.free(&c, int_ptr(s), (int32_t)s->size(0), stream_of(dev)));
}

// Weights of a cache's sequences: float32 (layers, sequences, tokens), rows of their own.
bool weights_of(const Tensor *t, int device, const attn_cache &c, attn_weights &w) {
    if (!on(t, device) || t->dim() != 3 || t->scalar_type() != at::kFloat || t->size(0) < 1 || t->size(1) != c.max_seqs ||
        !fits(t->size(0)) || !fits(t->size(2)) || (t->size(2) > 1 && t->stride(2) != 1))
        return false;
    w.stride_seq = t->size(1) > 1 ? t->stride(1) : t->size(2);
    w.stride_layer = t->size(0) > 1 ? t->stride(0) : t->size(1) * t->size(2);
    if (w.stride_seq < t->size(2) || (t->size(0) > 1 && w.stride_layer < w.stride_seq * (t->size(1) - 1) + t->size(2)))
        return false;
    w.ptr = static_cast<float *>(t->data_ptr());
    w.n_layers = (int32_t)t->size(0);
    w.cols = (int32_t)t->size(2);
    return true;
}

// weigh(cache, device, seqs, cu, q, lse, weights, layer, scale, window, sinks, fresh) -> status | None
PyObject *py_weigh(PyObject *, PyObject *const *args, Py_ssize_t n) {
    attn_weigh_args a;
    std::memset(&a, 0, sizeof(a));
    attn_weights w;
    int dev;
    NEED(n == 12 && cache_of(args[0], args[1], a.cache, dev) && windowed(args[9], args[10], a.window, a.sinks));
    const Tensor *seqs = tensor(args[2]), *cu = tensor(args[3]), *q = tensor(args[4]), *lse = tensor(args[5]);
    long layer;
    NEED(ints(seqs, dev) && ints(cu, dev) && cu->size(0) == seqs->size(0) + 1 && fits(seqs->size(0)));
    NEED(q && rows(q, dev, a.cache.D, a.q) && dtype_code(*q) == a.cache.dtype && weights_of(tensor(args[6]), dev, a.cache, w) &&
         as_long(args[7], layer) && layer >= 0 && layer < a.cache.n_layers && layer < w.n_layers);
    const int64_t T = q->size(0), H = q->size(1);
    NEED(T > 0 && fits(T * H) && as_scale(args[8], a.cache.D, a.scale) && on(lse, dev) && lse->scalar_type() == at::kFloat &&
         lse->dim() == 2 && lse->size(0) == H && lse->size(1) == T && lse->is_contiguous());
    if (args[11] != Py_None) {
        const Tensor *fresh = tensor(args[11]);
        NEED(ints(fresh, dev) && fresh->size(0) == seqs->size(0));
        a.fresh = int_ptr(fresh);
    }
    a.layer = (int32_t)layer;
    a.H = (int32_t)H;
    a.lse = static_cast<const float *>(lse->data_ptr());
    a.weights = w.ptr + layer * w.stride_layer;
    a.weights_stride = w.stride_seq;
    a.cols = w.cols;
    a.n = (int32_t)seqs->size(0);
    a.n_q = (int32_t)T;
    a.seqs = int_ptr(seqs);
    a.cu = int_ptr(cu);
    const size_t bytes = api.weigh_bytes(&a);
    Tensor ws;
    if (bytes) {
        ws = scratch(bytes, dev);
        a.workspace = ws.data_ptr();
        a.workspace_bytes = (size_t)ws.size(0);
    }
    return status(api.weigh(&a, stream_of(dev)));
}

// evict(cache, device, seqs, budgets, weights, sinks, recent) -> status | None
PyObject *py_evict(PyObject *, PyObject *const *args, Py_ssize_t n) {
    attn_cache c;
    attn_weights w;
    int dev;
    NEED(n == 7 && cache_of(args[0], args[1], c, dev));
    const Tensor *s = tensor(args[2]), *b = tensor(args[3]);
    long sinks, recent;
    NEED(ints(s, dev) && ints(b, dev) && b->size(0) == s->size(0) && fits(s->size(0)) && weights_of(tensor(args[4]), dev, c, w));
    NEED(!PyBool_Check(args[5]) && !PyBool_Check(args[6]) && as_long(args[5], sinks) && as_long(args[6], recent) && sinks >= 0 &&
         recent >= 0);
    const Tensor ws = scratch(api.evict_bytes(&c, (int32_t)s->size(0), w.cols), dev);
    return status(api.evict(&c, int_ptr(s), int_ptr(b), (int32_t)s->size(0), &w, (int32_t)sinks, (int32_t)recent,
                            ws.data_ptr(), (size_t)ws.size(0), stream_of(dev)));
}

// init(addresses): the entry points, in Api's order
PyObject *py_init(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 1 || !PyTuple_Check(args[0]) || (size_t)PyTuple_GET_SIZE(args[0]) * sizeof(void *) != sizeof(api)) {
        PyErr_SetString(PyExc_TypeError, "init: one address per entry point");
        return nullptr;
    }
    void *at[sizeof(api) / sizeof(void *)];
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(args[0]); ++i) {
        at[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(args[0], i));
        if (!at[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "init: a null address");
            return nullptr;
        }
    }
    std::memcpy(&api, at, sizeof(api));
    Py_RETURN_NONE;
}

// No C++ exception (torch's allocator can throw) leaves an entry.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *args, Py_ssize_t n) {
    try {
        return F(self, args, n);
    } catch (const c10::OutOfMemoryError &) {
        Py_RETURN_NONE;  // the Python path allocates the same and raises torch's own exception
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

#define ENTRY(name, fn) \
    {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<fn>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    ENTRY("init", py_init),          ENTRY("fwd", py_fwd),
    ENTRY("bwd", py_bwd),            ENTRY("tree", py_tree),
    ENTRY("write", py_write),        ENTRY("extend", py_alloc<false>),
    ENTRY("fork", py_alloc<true>),   ENTRY("keep", py_keep),
    ENTRY("free", py_free),          ENTRY("weigh", py_weigh),
    ENTRY("evict", py_evict),        {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
