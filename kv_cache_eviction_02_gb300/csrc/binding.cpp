// Python module _binding: the tensor arguments of the shared-prompt decoding calls, which are made once
// per layer and decoded token. Each function checks every tensor against the declared shape (CUDA, on the
// call's device, of the element type, large enough, contiguous or with rows a stride apart) and calls the
// C-ABI, for which it takes under a microsecond; the same checks through ctypes and tensor attributes cost
// more than the launches (7 us of a 14 us pg_attention call). A call whose arguments do not fit, or are
// addresses, returns kOther and touches nothing: the caller finds out what is wrong.
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/autograd/python_variable.h>

#include "kvevict.h"

namespace {

constexpr long kOther = -1;

decltype(&pg_plan) g_plan;
decltype(&pg_append) g_append;
decltype(&pg_attention) g_attention;

struct Args {
    PyObject *const *at;
    const KvePgShape *shape;
    c10::DeviceIndex device;
    void *stream;
    at::ScalarType type;
    bool ok = true;

    Args(PyObject *const *args) : at(args + 3) {
        shape = static_cast<const KvePgShape *>(PyLong_AsVoidPtr(args[0]));
        const long dev = PyLong_AsLong(args[1]);
        stream = PyLong_AsVoidPtr(args[2]);
        ok = shape && dev >= 0 && dev < 128 && !PyErr_Occurred();
        device = static_cast<c10::DeviceIndex>(dev);
        if (ok)
            type = shape->dtype == KVE_F32 ? at::kFloat
                                           : (shape->dtype == KVE_BF16 ? at::kBFloat16 : at::kHalf);
    }
    const at::Tensor *tensor(int i, at::ScalarType t) {
        if (!ok || !THPVariable_Check(at[i])) return ok = false, nullptr;
        const at::Tensor &x = THPVariable_Unpack(at[i]);
        if (x.scalar_type() != t || !x.is_cuda() || x.get_device() != device) return ok = false, nullptr;
        return &x;
    }
    // a contiguous array; with `none` it may be missing
    template <typename T = void> T *array(int i, at::ScalarType t, long long numel, bool none = false) {
        if (at[i] == Py_None) {
            ok = ok && none;
            return nullptr;
        }
        const at::Tensor *x = tensor(i, t);
        if (!x) return nullptr;
        if (x->numel() < numel || !x->is_contiguous()) return ok = false, nullptr;
        return static_cast<T *>(x->data_ptr());
    }
    int32_t *ints(int i, long long numel, bool none = false) {
        return array<int32_t>(i, at::kInt, numel, none);
    }
    // packed rows [n_rows][heads][d_head] that may lie apart
    const void *rows(int i, int heads, long long *stride) {
        const int n = ok ? shape->n_rows : 0, d = ok ? shape->d_head : 0;
        *stride = (long long)heads * d;
        const at::Tensor *x = tensor(i, type);
        if (!x) return nullptr;
        if (x->dim() != 3 || x->size(1) != heads || x->size(2) != d)
            return array(i, type, (long long)n * heads * d);
        if (x->size(0) < n || (d > 1 && x->stride(2) != 1) || (heads > 1 && x->stride(1) != d))
            return ok = false, nullptr;
        if (n > 1) *stride = x->stride(0);
        return x->data_ptr();
    }
    // a prompt cache [n_prompts][n_kv_heads][>= n_prefix][d_head]
    const void *prefix(int i, long long (&s)[3]) {
        if (!ok) return nullptr;
        const long long S = shape->n_prompts, H = shape->n_kv_heads, n = shape->n_prefix, d = shape->d_head;
        s[0] = H * n * d;
        s[1] = n * d;
        s[2] = d;
        if (at[i] == Py_None) return nullptr;
        const at::Tensor *x = tensor(i, type);
        if (!x) return nullptr;
        if (x->dim() != 4) return array(i, type, S * H * n * d);
        if (x->size(0) != S || x->size(1) != H || x->size(2) < n || x->size(3) != d ||
            (d > 1 && x->stride(3) != 1))
            return ok = false, nullptr;
        for (int k = 0; k < 3; ++k) s[k] = x->stride(k);
        return x->data_ptr();
    }
    long long requests() const { return ok ? (long long)shape->n_prompts * shape->fan : 0; }
    long long pool() const {
        return ok ? (long long)shape->n_pages * shape->n_kv_heads * shape->page_size * shape->d_head : 0;
    }
};

template <typename F> PyObject *result(Args &a, F call) {
    if (!a.ok) {
        PyErr_Clear();
        return PyLong_FromLong(kOther);
    }
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = call();
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(status);
}

// No exception leaves a function: tensors without storage throw when asked for their address.
template <PyObject *(*F)(Args &), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N + 3) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        Args a(args);
        return F(a);
    } catch (...) {
        PyErr_Clear();
        return PyLong_FromLong(kOther);
    }
}

PyObject *plan(Args &a) {
    const long long R = a.requests(), n = a.ok ? a.shape->n_rows : 0;
    const int32_t *new_len = a.ints(0, R), *len_in = a.ints(1, R), *pool_in = a.ints(2, 4);
    int32_t *free_pages = a.ints(3, a.ok ? a.shape->n_pages : 0);
    int32_t *table = a.ints(4, a.ok ? R * a.shape->max_pages : 0);
    int32_t *len_out = a.ints(5, R), *pool_out = a.ints(6, 4), *q_start = a.ints(7, R + 1);
    int32_t *row_req = a.ints(8, n), *row_pos = a.ints(9, n), *slots = a.ints(10, n);
    return result(a, [&] {
        return g_plan(a.shape, new_len, len_in, pool_in, free_pages, table, len_out, pool_out, q_start,
                      row_req, row_pos, slots, a.stream);
    });
}

PyObject *append(Args &a) {
    const int heads = a.ok ? a.shape->n_kv_heads : 0;
    long long ks, vs;
    const void *k = a.rows(0, heads, &ks), *v = a.rows(1, heads, &vs);
    const int32_t *slots = a.ints(2, a.ok ? a.shape->n_rows : 0);
    void *K = a.array(3, a.type, a.pool()), *V = a.array(4, a.type, a.pool());
    return result(a, [&] { return g_append(a.shape, k, v, ks, vs, slots, K, V, a.stream); });
}

PyObject *attention(Args &a) {
    const long long R = a.requests(), n = a.ok ? a.shape->n_rows : 0;
    const long long heads = a.ok ? n * a.shape->n_q_heads : 0;
    long long qs, s[3], t[3];
    const void *q = a.rows(0, a.ok ? a.shape->n_q_heads : 0, &qs);
    const void *Kp = a.prefix(1, s), *Vp = a.prefix(2, t);
    a.ok = a.ok && s[0] == t[0] && s[1] == t[1] && s[2] == t[2];
    const int32_t *plen = a.ints(3, a.ok ? a.shape->n_prompts : 0, true);
    const void *K = a.array(4, a.type, a.pool()), *V = a.array(5, a.type, a.pool());
    const int32_t *table = a.ints(6, a.ok ? R * a.shape->max_pages : 0), *len = a.ints(7, R);
    const int32_t *q_start = a.ints(8, R + 1), *row_req = a.ints(9, n);
    void *out = a.array(10, a.type, a.ok ? heads * a.shape->d_head : 0);
    float *lse = a.array<float>(11, at::kFloat, heads, true);
    void *ws = nullptr;
    size_t bytes = 0;
    if (a.ok && a.at[12] != Py_None) {
        a.ok = THPVariable_Check(a.at[12]);
        if (a.ok) {
            const at::Tensor &x = THPVariable_Unpack(a.at[12]);
            a.ok = x.is_cuda() && x.get_device() == a.device && x.is_contiguous();
            if (a.ok) {
                ws = x.data_ptr();
                bytes = x.nbytes();
            }
        }
    }
    return result(a, [&] {
        return g_attention(a.shape, q, qs, Kp, Vp, s[0], s[1], s[2], plen, K, V, table, len, q_start,
                           row_req, out, lse, ws, bytes, a.stream);
    });
}

// the addresses of pg_plan, pg_append and pg_attention in the library that the package has loaded
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 3) {
        PyErr_SetString(PyExc_TypeError, "three addresses");
        return nullptr;
    }
    g_plan = reinterpret_cast<decltype(g_plan)>(PyLong_AsVoidPtr(args[0]));
    g_append = reinterpret_cast<decltype(g_append)>(PyLong_AsVoidPtr(args[1]));
    g_attention = reinterpret_cast<decltype(g_attention)>(PyLong_AsVoidPtr(args[2]));
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef methods[] = {
    {"bind", FAST(&bind), METH_FASTCALL, nullptr},
    {"plan", FAST((&entry<plan, 11>)), METH_FASTCALL, nullptr},
    {"append", FAST((&entry<append, 5>)), METH_FASTCALL, nullptr},
    {"attention", FAST((&entry<attention, 13>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module{PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr,
                   nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
