// binding.cpp -- the Python side of the paged cache's calls: reads the tensors
// of one call, checks that they fit together and calls the C entry point.
//
// A decode step makes these calls once or twice per layer with about ten tensors
// each; asking every tensor for its type, device, shape, strides and address from
// Python costs more than the launch (mnb_rope_append: 6.5 us of 10.4).  Each
// function returns the C call's status, or None when the tensors do not fit
// together: the caller then works out what is wrong and raises.  No arithmetic
// and no CUDA code is here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mnb.h"

namespace {

// What the checks of one call need, and whether all of them have passed.
struct Call {
    int dev = -1;
    bool ok = true;

    const at::Tensor *tensor(PyObject *o) {
        if (!THPVariable_Check(o)) {
            ok = false;
            return nullptr;
        }
        return &THPVariable_Unpack(o);
    }

    // `n` contiguous elements of type t (n < 0: any number); their address.
    void *flat(PyObject *o, at::ScalarType t, int64_t n) {
        const at::Tensor *x = tensor(o);
        if (!x || x->scalar_type() != t || !x->is_contiguous() || x->get_device() != dev || (n >= 0 && x->numel() != n)) {
            ok = false;
            return nullptr;
        }
        return const_cast<void *>(x->const_data_ptr());
    }
    void *flat_or_none(PyObject *o, at::ScalarType t, int64_t n) { return o == Py_None ? nullptr : flat(o, t, n); }

    // [n, heads, D] with a contiguous last dimension; address, row and head stride.
    void *rows(PyObject *o, at::ScalarType t, int64_t n, int64_t heads, int64_t D, int64_t *row, int64_t *head) {
        const at::Tensor *x = tensor(o);
        if (!x || x->scalar_type() != t || x->get_device() != dev || x->dim() != 3 || x->size(0) != n ||
            x->size(1) != heads || x->size(2) != D || (x->stride(2) != 1 && D > 1 && x->numel() > 0)) {
            ok = false;
            return nullptr;
        }
        *row = x->stride(0), *head = x->stride(1);
        return const_cast<void *>(x->const_data_ptr());
    }

    // Two pools [pages, page_size, heads, D] of one layout; sets the call's device.
    at::ScalarType pools(PyObject *ko, PyObject *vo, mnb_paged_cache *c) {
        const at::Tensor *k = tensor(ko), *v = tensor(vo);
        if (!k || !v)
            return at::kHalf;
        const at::ScalarType t = k->scalar_type();
        dev = k->get_device();
        if ((t != at::kHalf && t != at::kFloat) || v->scalar_type() != t || k->dim() != 4 || v->sizes() != k->sizes() ||
            v->strides() != k->strides() || v->get_device() != dev || dev < 0 || dev != c10::cuda::current_device() ||
            (k->stride(3) != 1 && k->size(3) > 1)) {
            ok = false;
            return t;
        }
        *c = {const_cast<void *>(k->const_data_ptr()), const_cast<void *>(v->const_data_ptr()), k->size(0), k->size(1),
              k->size(2), k->size(3), k->stride(0), k->stride(1), k->stride(2), t == at::kHalf ? MNB_F16 : MNB_F32, 0};
        return t;
    }

    // Rows of a block table [n, blocks]: address, row stride, blocks.
    int32_t *table(PyObject *o, int64_t n, int64_t *stride, int64_t *blocks) {
        const at::Tensor *x = tensor(o);
        if (!x || x->scalar_type() != at::kInt || x->get_device() != dev || x->dim() != 2 || x->size(0) != n ||
            (x->stride(1) != 1 && x->size(1) > 1 && n > 0)) {
            ok = false;
            return nullptr;
        }
        *blocks = x->size(1);
        *stride = n > 1 ? x->stride(0) : x->size(1);
        return static_cast<int32_t *>(const_cast<void *>(x->const_data_ptr()));
    }
};

int64_t whole(PyObject *o) { return PyLong_AsLongLong(o); }

// The C call, without the interpreter's lock: a launch may wait for room in the stream's queue.
template <typename Args>
PyObject *run(int (*fn)(const Args *, unsigned, void *), const Args &a, PyObject *flags, PyObject *stream, int dev) {
    const unsigned long f = PyLong_AsUnsignedLong(flags);
    void *s = stream == Py_None ? c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream()
                                : reinterpret_cast<void *>(PyLong_AsUnsignedLongLong(stream));
    if (PyErr_Occurred())
        return nullptr;
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = fn(&a, (unsigned)f, s);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

// Calls body(); what torch throws (a tensor without strides, say) counts as a failed check.
template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F body) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", n, want);
        return nullptr;
    }
    try {
        return body();
    } catch (...) {
        if (PyErr_Occurred())
            return nullptr;
        Py_RETURN_NONE;
    }
}

PyObject *paged_tables(PyObject *, PyObject *const *p, Py_ssize_t n) {
    return guarded(n, 15, [&]() -> PyObject * {
        Call c;
        mnb_paged_tables_args a = {};
        const at::Tensor *ctx = c.tensor(p[0]), *slots = c.tensor(p[8]), *free_pages = c.tensor(p[5]);
        if (!c.ok)
            Py_RETURN_NONE;
        c.dev = ctx->get_device();
        c.ok = c.dev >= 0 && c.dev == c10::cuda::current_device();
        a.B = ctx->numel(), a.T = slots->numel(), a.num_free = free_pages->numel();
        a.ctx_lens = (int32_t *)c.flat(p[0], at::kInt, a.B);
        a.new_lens = (int32_t *)c.flat(p[1], at::kInt, a.B);
        a.block_table = c.table(p[2], a.B, &a.table_stride, &a.max_blocks);
        a.page_size = whole(p[3]), a.num_pages = whole(p[4]);
        a.free_pages = (int32_t *)c.flat(p[5], at::kInt, a.num_free);
        a.free_start = (int32_t *)c.flat(p[6], at::kInt, 1);
        a.seq_lens = (int32_t *)c.flat(p[7], at::kInt, a.B);
        a.slots = (int32_t *)c.flat(p[8], at::kInt, a.T);
        a.positions = (int32_t *)c.flat(p[9], at::kInt, a.T);
        a.cu_new = (int32_t *)c.flat(p[10], at::kInt, a.B + 1);
        a.free_next = (int32_t *)c.flat(p[11], at::kInt, 1);
        a.status = (int *)c.flat_or_none(p[12], at::kInt, 1);
        if (PyErr_Occurred())
            return nullptr;
        if (!c.ok)
            Py_RETURN_NONE;
        return run(mnb_paged_tables, a, p[13], p[14], c.dev);
    });
}

PyObject *rope_append(PyObject *, PyObject *const *p, Py_ssize_t n) {
    return guarded(n, 16, [&]() -> PyObject * {
        Call c;
        mnb_rope_append_args a = {};
        const at::ScalarType t = c.pools(p[3], p[4], &a.cache);
        const at::Tensor *slots = c.tensor(p[5]);
        if (!c.ok)
            Py_RETURN_NONE;
        const int64_t H = a.cache.num_heads, D = a.cache.head_dim;
        a.T = slots->numel();
        a.slots = (int32_t *)c.flat(p[5], at::kInt, a.T);
        a.positions = (int32_t *)c.flat_or_none(p[6], at::kInt, a.T);
        if (p[0] != Py_None) {
            const at::Tensor *q = c.tensor(p[0]);
            a.Hq = q && q->dim() == 3 ? q->size(1) : -1;
            a.q = c.rows(p[0], t, a.T, a.Hq, D, &a.q_token_stride, &a.q_head_stride);
            a.q_out = c.rows(p[9], t, a.T, a.Hq, D, &a.o_token_stride, &a.o_head_stride);
        }
        a.k = c.rows(p[1], t, a.T, H, D, &a.k_token_stride, &a.k_head_stride);
        a.v = c.rows(p[2], t, a.T, H, D, &a.v_token_stride, &a.v_head_stride);
        if (p[7] != Py_None) {
            const at::Tensor *cos = c.tensor(p[7]), *sin = c.tensor(p[8]);
            if (!c.ok || cos->dim() != 2 || sin->sizes() != cos->sizes())
                Py_RETURN_NONE;
            a.num_pos = cos->size(0), a.rot_dim = 2 * cos->size(1);
            a.cos = (float *)c.flat(p[7], at::kFloat, -1);
            a.sin = (float *)c.flat(p[8], at::kFloat, -1);
        }
        a.q_weight = (float *)c.flat_or_none(p[10], at::kFloat, D);
        a.k_weight = (float *)c.flat_or_none(p[11], at::kFloat, D);
        a.eps = (float)PyFloat_AsDouble(p[12]);
        a.status = (int *)c.flat_or_none(p[13], at::kInt, 1);
        if (PyErr_Occurred())
            return nullptr;
        if (!c.ok)
            Py_RETURN_NONE;
        return run(mnb_rope_append, a, p[14], p[15], c.dev);
    });
}

PyObject *paged_attention(PyObject *, PyObject *const *p, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject * {
        Call c;
        mnb_paged_attention_args a = {};
        const at::ScalarType t = c.pools(p[1], p[2], &a.cache);
        const at::Tensor *q = c.tensor(p[0]), *ws = c.tensor(p[7]);
        if (!c.ok || q->dim() != 3)
            Py_RETURN_NONE;
        const int64_t D = a.cache.head_dim;
        a.B = q->size(0), a.Hq = q->size(1);
        a.q = c.rows(p[0], t, a.B, a.Hq, D, &a.q_request_stride, &a.q_head_stride);
        a.block_table = c.table(p[3], a.B, &a.table_stride, &a.max_blocks);
        a.seq_lens = (int32_t *)c.flat(p[4], at::kInt, a.B);
        a.scale = (float)PyFloat_AsDouble(p[5]);
        a.out = c.rows(p[6], t, a.B, a.Hq, D, &a.o_request_stride, &a.o_head_stride);
        a.workspace = c.flat(p[7], at::kByte, -1);
        a.ws_bytes = (size_t)ws->numel();
        a.lse = (float *)c.flat_or_none(p[8], at::kFloat, a.B * a.Hq);
        a.status = (int *)c.flat_or_none(p[9], at::kInt, 1);
        if (PyErr_Occurred())
            return nullptr;
        if (!c.ok)
            Py_RETURN_NONE;
        return run(mnb_paged_attention, a, p[10], p[11], c.dev);
    });
}

PyMethodDef methods[] = {
    {"paged_tables", (PyCFunction)(void (*)(void))paged_tables, METH_FASTCALL, nullptr},
    {"rope_append", (PyCFunction)(void (*)(void))rope_append, METH_FASTCALL, nullptr},
    {"paged_attention", (PyCFunction)(void (*)(void))paged_attention, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch that the calls above were compiled against, whose C++ classes they use.
PyMODINIT_FUNC PyInit__binding(void) {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", MNB_TORCH) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
