// Argument marshalling of the quantised-cache and page calls for Python, natively: a call whose
// kernel runs a few microseconds is otherwise bound by interpreted checks (8.9 us for an append of
// 12 arguments through ctypes; the library's own part, checks and launch, is 2.7 us).
//
// Each function checks types, shapes and contiguity of its tensors, takes the current stream and
// calls libdsa.  It returns the call's status, or -1 without calling anything when an argument
// is not what the call takes: the binding then names the argument in its own checks.
#include <Python.h>

#include <dlfcn.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/dsa.h"

namespace {

#define DSA_CALLS(X)                                                                                      \
    X(dsa_kv_append_quant) X(dsa_sparse_attn_decode_quant) X(dsa_sparse_attn_prefill_quant)               \
    X(dsa_window_attn_quant) X(dsa_pages_fork) X(dsa_pages_fork_workspace_size) X(dsa_pages_release)      \
    X(dsa_pages_compact) X(dsa_pages_compact_workspace_size)

struct Library {
#define X(f) decltype(&::f) f = nullptr;
    DSA_CALLS(X)
#undef X
} lib;

struct Refused {};                                   // an argument the binding has to look at

const at::Tensor &tensor(PyObject *o, at::ScalarType type)
{
    if (!THPVariable_Check(o)) throw Refused();
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.scalar_type() != type || !t.is_cuda() || !t.is_contiguous()) throw Refused();
    return t;
}

const at::Tensor &tensor(PyObject *o, at::ScalarType type, at::IntArrayRef shape)
{
    const at::Tensor &t = tensor(o, type);
    if (t.sizes() != shape) throw Refused();
    return t;
}

template <typename T>
T *ptr(const at::Tensor &t) { return static_cast<T *>(t.data_ptr()); }

int32_t *int_or_null(PyObject *o, int64_t n) { return o == Py_None ? nullptr : ptr<int32_t>(tensor(o, at::kInt, {n})); }

dsa_stream_t stream() { return reinterpret_cast<dsa_stream_t>(c10::cuda::getCurrentCUDAStream().stream()); }

int32_t count(int64_t n)
{
    if (n > INT32_MAX) throw Refused();
    return (int32_t)n;
}

// Runs f (no Python object touched), with the interpreter free for other threads.
template <typename F>
PyObject *call(F f)
{
    long st;
    Py_BEGIN_ALLOW_THREADS
    st = (long)f();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F f)
{
    if (n != want || !lib.dsa_kv_append_quant) return PyLong_FromLong(-1);
    try {
        return f();
    } catch (...) {                                  // a tensor without storage, an allocation that failed, ...
        PyErr_Clear();
        return PyLong_FromLong(-1);
    }
}

struct Cache {
    uint8_t *codes;
    float *scale;
    int64_t n_pages;
    const int32_t *table;
    int n_req, max_pages;
    Cache(PyObject *c, PyObject *s, PyObject *t)
    {
        const at::Tensor &codes_t = tensor(c, at::kByte);
        if (codes_t.dim() != 6) throw Refused();
        n_pages = codes_t.size(0);
        if (codes_t.sizes() != at::IntArrayRef({n_pages, 4, 8, 2, 8, 192})) throw Refused();
        codes = ptr<uint8_t>(codes_t);
        scale = ptr<float>(tensor(s, at::kFloat, {n_pages, 4, 8, 2}));
        const at::Tensor &table_t = tensor(t, at::kInt);
        if (table_t.dim() != 2) throw Refused();
        n_req = count(table_t.size(0));
        max_pages = count(table_t.size(1));
        table = ptr<int32_t>(table_t);
    }
};

// kv_cache, kv_scale, block_table, q_pos, new_k, new_v, q_req
PyObject *kv_append_quant(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 7, [&] {
        const Cache c(a[0], a[1], a[2]);
        const at::Tensor &pos = tensor(a[3], at::kInt);
        if (pos.dim() != 1) throw Refused();
        const int64_t m = pos.size(0);
        const void *nk = ptr<void>(tensor(a[4], at::kBFloat16, {m, 4, 192}));
        const void *nv = ptr<void>(tensor(a[5], at::kBFloat16, {m, 4, 192}));
        const int32_t *req = int_or_null(a[6], m);
        if (!req && m > c.n_req) throw Refused();
        const int32_t *p = ptr<int32_t>(pos);
        const int tokens = count(m);
        const dsa_stream_t st = stream();
        return call([&] {
            return lib.dsa_kv_append_quant(c.codes, c.scale, c.n_pages, c.table, c.max_pages, c.n_req, req, p, tokens, nk,
                                           nv, st);
        });
    });
}

// q, kv_cache, kv_scale, block_table, q_req (None: identity), q_pos, sel_idx, sel_count (None: the window),
// window, out, lse
PyObject *attn_quant(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 11, [&] {
        const at::Tensor &q = tensor(a[0], at::kBFloat16);
        if (q.dim() != 3) throw Refused();
        const int64_t nq = q.size(0);
        if (q.size(1) != 64 || q.size(2) != 192) throw Refused();
        const Cache c(a[1], a[2], a[3]);
        const int32_t *req = int_or_null(a[4], nq);
        if (!req && nq > c.n_req) throw Refused();
        const int32_t *pos = ptr<int32_t>(tensor(a[5], at::kInt, {nq}));
        const bool selected = a[6] != Py_None;
        const int32_t *sel = nullptr, *cnt = nullptr;
        int k = 0, window = 0;
        if (selected) {
            const at::Tensor &s = tensor(a[6], at::kInt);
            if (s.dim() != 3 || s.size(0) != nq || s.size(1) != 4) throw Refused();
            k = count(s.size(2));
            sel = ptr<int32_t>(s);
            cnt = ptr<int32_t>(tensor(a[7], at::kInt, {nq, 4}));
        } else {
            window = count(PyLong_AsLongLong(a[8]));
            if (PyErr_Occurred() || window < 0) throw Refused();
        }
        void *out = ptr<void>(tensor(a[9], at::kBFloat16, {nq, 64, 192}));
        float *lse = a[10] == Py_None ? nullptr : ptr<float>(tensor(a[10], at::kFloat, {nq, 64}));
        const void *qp = ptr<void>(q);
        const int m = count(nq);
        const dsa_stream_t st = stream();
        if (!selected)
            return call([&] {
                return lib.dsa_window_attn_quant(qp, c.codes, c.scale, c.n_pages, c.table, c.max_pages, c.n_req, req, pos, m,
                                                 window, out, lse, st);
            });
        if (!req)
            return call([&] {
                return lib.dsa_sparse_attn_decode_quant(qp, c.codes, c.scale, c.n_pages, c.table, c.max_pages, pos, m, sel,
                                                        cnt, k, out, lse, st);
            });
        return call([&] {
            return lib.dsa_sparse_attn_prefill_quant(qp, c.codes, c.scale, c.n_pages, c.table, c.max_pages, c.n_req, req, pos,
                                                     m, sel, cnt, k, out, lse, st);
        });
    });
}

struct Tables {
    const int32_t *ref, *table;
    int32_t *ref_out, *table_out;
    int64_t n_pages;
    int n_req, max_pages;
    at::TensorOptions bytes;                         // of a workspace beside them
    Tables(PyObject *r, PyObject *t, PyObject *ro, PyObject *to)
    {
        const at::Tensor &rt = tensor(r, at::kInt), &tt = tensor(t, at::kInt);
        if (rt.dim() != 1 || tt.dim() != 2) throw Refused();
        n_pages = rt.size(0);
        n_req = count(tt.size(0));
        max_pages = count(tt.size(1));
        ref = ptr<int32_t>(rt);
        table = ptr<int32_t>(tt);
        ref_out = ptr<int32_t>(tensor(ro, at::kInt, rt.sizes()));
        table_out = ptr<int32_t>(tensor(to, at::kInt, tt.sizes()));
        bytes = rt.options().dtype(at::kByte);
    }
};

struct Pools {
    dsa_page_pool_t pool[DSA_MAX_PAGE_POOLS];
    int n;
    Pools(PyObject *list, int64_t n_pages)
    {
        if (!PyList_Check(list) && !PyTuple_Check(list)) throw Refused();
        const Py_ssize_t m = PySequence_Fast_GET_SIZE(list);
        if (m > DSA_MAX_PAGE_POOLS) throw Refused();
        n = (int)m;
        for (int i = 0; i < n; ++i) {
            PyObject *o = PySequence_Fast_GET_ITEM(list, i);
            if (!THPVariable_Check(o)) throw Refused();
            const at::Tensor &t = THPVariable_Unpack(o);
            if (!t.is_cuda() || !t.is_contiguous() || t.dim() < 2 || t.size(0) != n_pages) throw Refused();
            pool[i].data = t.data_ptr();
            pool[i].page_bytes = n_pages > 0 ? t.numel() / n_pages * (int64_t)t.element_size() : 0;
        }
    }
};

// ref, block_table, parent, child, length, pools, ref_out, table_out
PyObject *pages_fork(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 8, [&] {
        const Tables t(a[0], a[1], a[6], a[7]);
        const at::Tensor &parent = tensor(a[2], at::kInt);
        if (parent.dim() != 1) throw Refused();
        const int64_t m = parent.size(0);
        const int32_t *c = ptr<int32_t>(tensor(a[3], at::kInt, {m})), *l = ptr<int32_t>(tensor(a[4], at::kInt, {m}));
        const Pools p(a[5], t.n_pages);
        const int forks = count(m);
        const size_t need = lib.dsa_pages_fork_workspace_size(forks);
        at::Tensor ws = at::empty({(int64_t)need}, t.bytes);
        const int32_t *pr = ptr<int32_t>(parent);
        void *w = need ? ws.data_ptr() : nullptr;
        const dsa_stream_t st = stream();
        return call([&] {
            return lib.dsa_pages_fork(t.ref, t.ref_out, t.n_pages, t.table, t.table_out, t.max_pages, t.n_req, pr, c, l, forks,
                                      p.pool, p.n, w, need, st);
        });
    });
}

// ref, block_table, req, keep, ref_out, table_out
PyObject *pages_release(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 6, [&] {
        const Tables t(a[0], a[1], a[4], a[5]);
        const at::Tensor &req = tensor(a[2], at::kInt);
        if (req.dim() != 1) throw Refused();
        const int32_t *keep = ptr<int32_t>(tensor(a[3], at::kInt, req.sizes())), *r = ptr<int32_t>(req);
        const int m = count(req.size(0));
        const dsa_stream_t st = stream();
        return call([&] {
            return lib.dsa_pages_release(t.ref, t.ref_out, t.n_pages, t.table, t.table_out, t.max_pages, t.n_req, r, keep, m,
                                         st);
        });
    });
}

// ref, block_table, pools, ref_out, table_out, new_index, n_live
PyObject *pages_compact(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 7, [&] {
        const Tables t(a[0], a[1], a[3], a[4]);
        const Pools p(a[2], t.n_pages);
        int32_t *index = ptr<int32_t>(tensor(a[5], at::kInt, {t.n_pages})), *live = ptr<int32_t>(tensor(a[6], at::kInt, {1}));
        const size_t need = lib.dsa_pages_compact_workspace_size(t.n_pages);
        at::Tensor ws = at::empty({(int64_t)need}, t.bytes);
        void *w = need ? ws.data_ptr() : nullptr;
        const dsa_stream_t st = stream();
        return call([&] {
            return lib.dsa_pages_compact(t.ref, t.ref_out, t.n_pages, t.table, t.table_out, t.max_pages, t.n_req, index, live,
                                         p.pool, p.n, w, need, st);
        });
    });
}

// bind(path): takes the calls from the library at `path`.
PyObject *bind(PyObject *, PyObject *path)
{
    const char *file = PyUnicode_AsUTF8(path);
    if (!file) return nullptr;
    void *h = dlopen(file, RTLD_NOW | RTLD_LOCAL);
    if (!h) {
        PyErr_SetString(PyExc_ImportError, dlerror());
        return nullptr;
    }
    Library l;
#define X(f)                                                                      \
    l.f = reinterpret_cast<decltype(&::f)>(dlsym(h, #f));                         \
    if (!l.f) {                                                                   \
        PyErr_SetString(PyExc_ImportError, "libdsa has no " #f);                  \
        return nullptr;                                                           \
    }
    DSA_CALLS(X)
#undef X
    lib = l;
    Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(kv_append_quant), FAST(attn_quant), FAST(pages_fork), FAST(pages_release),
                         FAST(pages_compact), {"bind", bind, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", "Native argument marshalling of libdsa's calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
