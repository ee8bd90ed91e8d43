// Fast path of the Python binding for the calls of a decode step.
//
// The attention and cache calls take a few microseconds on the GPU; checking
// a dozen tensors from Python takes ten. Each function here takes the Python
// wrapper's arguments, checks that they are the plain case (tensors of the
// expected types, shapes and layouts on the current device, the current
// stream, outputs and workspace given) and makes the call. It returns the
// call's status, or None, having done nothing, if anything is not the plain
// case: the wrapper then goes through its own checks, which raise the errors.
// The address of the C entry point is the first argument.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <vector>

#include "jet.h"

namespace {

using at::Tensor;

struct Args {
    PyObject* const* a;
    int device = -1;
    at::ScalarType dt = at::kFloat;
    bool ok = true;

    const Tensor* tensor(int i) {
        if (!THPVariable_Check(a[i])) { ok = false; return nullptr; }
        return &THPVariable_Unpack(a[i]);
    }
    // a tensor of this type on the call's device
    const Tensor* on(int i, at::ScalarType t, int dim) {
        const Tensor* x = tensor(i);
        if (x && (!x->is_cuda() || x->get_device() != device || x->scalar_type() != t || x->dim() != dim)) ok = false;
        return x;
    }
    // contiguous, of this shape; the address
    void* dense(int i, at::ScalarType t, std::initializer_list<int64_t> shape) {
        const Tensor* x = on(i, t, (int)shape.size());
        if (!ok || !x) return nullptr;
        if (!x->is_contiguous() || x->sizes() != c10::IntArrayRef(shape.begin(), shape.size())) { ok = false; return nullptr; }
        return x->data_ptr();
    }
    void* dense_or_null(int i, at::ScalarType t, std::initializer_list<int64_t> shape) {
        return a[i] == Py_None ? nullptr : dense(i, t, shape);
    }
    // [N, heads, d] with dense rows of heads; the address and the elements between tokens
    void* rows(int i, int64_t N, int64_t H, int64_t d, int64_t& stride) {
        const Tensor* x = on(i, dt, 3);
        if (!ok || !x) return nullptr;
        const auto s = x->sizes(), st = x->strides();
        if (s[0] != N || s[1] != H || s[2] != d || st[2] != 1 || (H > 1 && st[1] != d)) { ok = false; return nullptr; }
        stride = N > 1 ? st[0] : H * d;
        return x->data_ptr();
    }
    // a call on this tensor's device and its current stream
    const Tensor* lead(int i) {
        const Tensor* q = tensor(i);
        if (!q || !q->is_cuda() || q->dim() < 2) { ok = false; return nullptr; }
        device = q->get_device();
        dt = q->scalar_type();
        if (device != c10::cuda::current_device()) ok = false;
        return q;
    }
    void* stream() const { return c10::cuda::getCurrentCUDAStream(device).stream(); }
    int64_t integer(int i) {
        const long long v = PyLong_AsLongLong(a[i]);
        if (v == -1 && PyErr_Occurred()) { PyErr_Clear(); ok = false; }
        return v;
    }
    double real(int i) {
        const double v = PyFloat_AsDouble(a[i]);
        if (v == -1.0 && PyErr_Occurred()) { PyErr_Clear(); ok = false; }
        return v;
    }
};

struct Pools {
    void *k = nullptr, *v = nullptr;
    int64_t st[3], n_pages = 0, page = 0, Hk = 0;
};

void kv_pools(Args& g, int ik, int iv, int64_t d, Pools& p) {
    const Tensor *k = g.on(ik, g.dt, 4), *v = g.on(iv, g.dt, 4);
    if (!g.ok || !k || !v) return;
    const auto s = k->sizes(), st = k->strides();
    if (s[3] != d || st[3] != 1 || v->sizes() != s || v->strides() != st) { g.ok = false; return; }
    for (int i = 0; i < 3; ++i) p.st[i] = s[i] > 1 ? st[i] : d;      // an axis of one entry has no stride that matters
    p.k = k->data_ptr();
    p.v = v->data_ptr();
    p.n_pages = s[0];
    p.Hk = s[1];
    p.page = s[2];
}

bool small(std::initializer_list<int64_t> xs) {
    for (int64_t x : xs)
        if (x < 0 || x > 0x7fffffff) return false;
    return true;
}

jet_dtype code(at::ScalarType t) { return t == at::kBFloat16 ? JET_BF16 : JET_F32; }
bool stored(at::ScalarType t) { return t == at::kBFloat16 || t == at::kFloat; }

PyObject* none() { Py_RETURN_NONE; }

// (address, q, k, v, q_gamma, k_gamma, inv_freq, cu_q, kv_lens, page_table, k_pool, v_pool, q_out, eps, interleaved)
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 15) return none();
    Args g{a};
    const auto fn = reinterpret_cast<decltype(&jet_attn_rope_append)>(g.integer(0));
    const Tensor* q = g.lead(1);
    if (!g.ok || q->dim() != 3 || !stored(g.dt)) return none();
    const int64_t N = q->size(0), Hq = q->size(1), d = q->size(2);
    Pools p;
    kv_pools(g, 10, 11, d, p);
    if (!g.ok) return none();
    int64_t qs, ks, vs, os;
    void *qp = g.rows(1, N, Hq, d, qs), *kp = g.rows(2, N, p.Hk, d, ks), *vp = g.rows(3, N, p.Hk, d, vs);
    void* op = g.rows(12, N, Hq, d, os);
    void *gq = g.dense_or_null(4, at::kFloat, {d}), *gk = g.dense_or_null(5, at::kFloat, {d});
    int64_t half = 0;
    void* fr = nullptr;
    if (a[6] != Py_None) {
        const Tensor* f = g.on(6, at::kFloat, 1);
        if (!g.ok || !f->is_contiguous()) return none();
        half = f->size(0);
        fr = f->data_ptr();
    }
    const Tensor* t = g.on(9, at::kInt, 2);
    if (!g.ok || !t->is_contiguous()) return none();
    const int64_t nseq = t->size(0), width = t->size(1);
    void *cu = g.dense(7, at::kInt, {nseq + 1}), *kl = g.dense(8, at::kInt, {nseq});
    const double eps = g.real(13);
    const int inter = PyObject_IsTrue(a[14]);
    if (!g.ok || inter < 0 || !small({N, nseq, width, p.n_pages, p.page, Hq, p.Hk, d, 2 * half})) return none();
    void* s = g.stream();
    jet_status st;
    Py_BEGIN_ALLOW_THREADS
    st = fn(qp, qs, kp, ks, vp, vs, (const float*)gq, (const float*)gk, (float)eps, (const float*)fr, (int)(2 * half), inter,
            op, os, p.k, p.v, p.st[0], p.st[1], p.st[2], (const int*)cu, (const int*)kl, t->data_ptr<int>(), (int)nseq,
            (int)N, (int)width, (int)p.n_pages, (int)p.page, (int)Hq, (int)p.Hk, (int)d, code(g.dt), s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

// (address, q, k_pool, v_pool, cu_q, kv_lens, page_table, max_new, o, workspace, window, scale)
PyObject* attn_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 12) return none();
    Args g{a};
    const auto fn = reinterpret_cast<decltype(&jet_attn_paged)>(g.integer(0));
    const Tensor* q = g.lead(1);
    if (!g.ok || q->dim() != 3 || !stored(g.dt)) return none();
    const int64_t N = q->size(0), Hq = q->size(1), d = q->size(2);
    Pools p;
    kv_pools(g, 2, 3, d, p);
    if (!g.ok) return none();
    int64_t qs;
    void *qp = g.rows(1, N, Hq, d, qs), *op = g.dense(8, g.dt, {N, Hq, d});
    const Tensor* t = g.on(6, at::kInt, 2);
    const Tensor* w = g.tensor(9);
    if (!g.ok || !t->is_contiguous() || !w->is_cuda() || w->get_device() != g.device || !w->is_contiguous()) return none();
    const int64_t nseq = t->size(0), width = t->size(1);
    void *cu = g.dense(4, at::kInt, {nseq + 1}), *kl = g.dense(5, at::kInt, {nseq});
    const int64_t max_new = g.integer(7), window = g.integer(10);
    const double scale = a[11] == Py_None ? std::pow((double)d, -0.5) : g.real(11);
    if (!g.ok || !small({N, nseq, width, p.n_pages, p.page, Hq, p.Hk, d, max_new, window})) return none();
    void* s = g.stream();
    jet_status st;
    Py_BEGIN_ALLOW_THREADS
    st = fn(qp, qs, p.k, p.v, p.st[0], p.st[1], p.st[2], (const int*)cu, (const int*)kl, t->data_ptr<int>(), op,
            w->data_ptr(), w->nbytes(), (int)nseq, (int)N, (int)max_new, (int)width, (int)p.n_pages, (int)p.page, (int)Hq,
            (int)p.Hk, (int)d, (int)window, (float)scale, code(g.dt), s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

// contiguous pools of equally many entries
struct Entries {
    std::vector<void*> base;
    std::vector<int64_t> bytes;
    int64_t n = 0;
};
bool entries(Args& g, PyObject* list, Entries& e) {
    if (!PyList_Check(list) || PyList_GET_SIZE(list) == 0) return false;
    const Py_ssize_t count = PyList_GET_SIZE(list);
    e.base.reserve(count);
    e.bytes.reserve(count);
    for (Py_ssize_t i = 0; i < count; ++i) {
        PyObject* item = PyList_GET_ITEM(list, i);
        if (!THPVariable_Check(item)) return false;
        const Tensor& t = THPVariable_Unpack(item);
        if (!t.is_cuda() || t.dim() < 2 || !t.is_contiguous()) return false;
        if (i == 0) {
            g.device = t.get_device();
            e.n = t.size(0);
            if (g.device != c10::cuda::current_device() || e.n <= 0) return false;
        }
        if (t.get_device() != g.device || t.size(0) != e.n) return false;
        e.base.push_back(t.data_ptr());
        e.bytes.push_back((int64_t)(t.nbytes() / (size_t)e.n));
    }
    return small({e.n});
}
bool indices(PyObject* list, std::vector<int>& out) {
    if (!PyList_Check(list)) return false;
    const Py_ssize_t n = PyList_GET_SIZE(list);
    out.reserve(n);
    for (Py_ssize_t i = 0; i < n; ++i) {
        PyObject* x = PyList_GET_ITEM(list, i);
        if (!PyLong_CheckExact(x)) return false;
        const long long v = PyLong_AsLongLong(x);
        if (v == -1 && PyErr_Occurred()) { PyErr_Clear(); return false; }
        if (v < 0 || v > 0x7fffffff) return false;
        out.push_back((int)v);
    }
    return true;
}

// (address, pools, src, dst)
PyObject* cache_copy(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 4) return none();
    Args g{a};
    const auto fn = reinterpret_cast<decltype(&jet_cache_copy)>(g.integer(0));
    Entries e;
    std::vector<int> src, dst;
    if (!g.ok || !entries(g, a[1], e) || !indices(a[2], src) || !indices(a[3], dst) || src.size() != dst.size())
        return none();
    void* s = g.stream();
    jet_status st;
    Py_BEGIN_ALLOW_THREADS
    st = fn(e.base.data(), e.bytes.data(), e.bytes.data(), (int)e.base.size(), (int)e.n, src.data(), dst.data(),
            (int)src.size(), s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

// (address, pools, page_table, kv_lens, page_size, page_table_out, n_live, workspace)
PyObject* cache_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 8) return none();
    Args g{a};
    const auto fn = reinterpret_cast<decltype(&jet_cache_compact)>(g.integer(0));
    Entries e;
    if (!g.ok || !entries(g, a[1], e)) return none();
    const Tensor* t = g.on(2, at::kInt, 2);
    const Tensor* w = g.tensor(7);
    if (!g.ok || !t->is_contiguous() || !w->is_cuda() || w->get_device() != g.device || !w->is_contiguous()) return none();
    const int64_t nseq = t->size(0), width = t->size(1), page = g.integer(4);
    void *kl = g.dense(3, at::kInt, {nseq}), *out = g.dense(5, at::kInt, {nseq, width}), *live = g.dense(6, at::kInt, {1});
    if (!g.ok || !small({nseq, width, page})) return none();
    void* s = g.stream();
    jet_status st;
    Py_BEGIN_ALLOW_THREADS
    st = fn(e.base.data(), e.bytes.data(), e.bytes.data(), (int)e.base.size(), (int)e.n, (int)page, t->data_ptr<int>(),
            (const int*)kl, (int)nseq, (int)width, (int*)out, (int*)live, w->data_ptr(), w->nbytes(), s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

// C++ exceptions (an allocation that fails) do not leave: the wrapper's own path then reports what is wrong
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    try {
        return F(self, a, n);
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}
#define ENTRY(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(guarded<f>)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {ENTRY(rope_append), ENTRY(attn_paged), ENTRY(cache_copy), ENTRY(cache_compact),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// `abi`: the torch and Python that it was compiled for, compared by the package before any call
PyMODINIT_FUNC PyInit__bind(void) {
    PyObject* m = PyModule_Create(&kModule);
    if (m && PyModule_AddStringConstant(m, "abi", JET_BIND_ABI) < 0) Py_CLEAR(m);
    return m;
}
