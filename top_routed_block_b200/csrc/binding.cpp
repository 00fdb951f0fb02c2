// binding.cpp -- the Python calls of the rotary positions and the 8-bit cache: takes torch
// tensors apart, checks their types, shapes and devices, allocates what the caller did
// not give, and calls the C ABI (include/fvattn.h).
//
// Why not ctypes, as for the other calls: these run for single tokens, where the GPU is
// done in a few microseconds.  fvattn_rope on [1, 2, 512, 64] took 29 us of host time through
// ctypes (18 us of Python around it, 3.6 us of converting 22 arguments); from here it takes
// 5.4, an append of one token 6.8, its attention 5.8 (two or three us of each are the launch).
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "fvattn.h"

namespace {

// Becomes Python's ValueError.
struct Refused : std::invalid_argument {
    using std::invalid_argument::invalid_argument;
};

[[noreturn]] void refuse(const char *what, const char *why) { throw Refused(std::string(what) + ": " + why); }

const at::Tensor &tensor(PyObject *o, const char *what) {
    if (!THPVariable_Check(o)) refuse(what, "expected a tensor");
    return THPVariable_Unpack(o);
}

// A bf16 tensor [B, H, n, d] with contiguous channels, and its strides (0 where there is one).
struct Heads {
    const void *ptr = nullptr;
    int64_t size[4] = {0, 0, 0, 0};
    int64_t stride[3] = {0, 0, 0};
    c10::Device device = c10::kCPU;

    bool like(const Heads &o) const { return std::equal(size, size + 4, o.size) && device == o.device; }
};

Heads heads_of(const at::Tensor &t, const char *what) {
    if (t.dim() != 4 || t.scalar_type() != at::kBFloat16 || !t.is_cuda())
        refuse(what, "expected a CUDA bf16 tensor [B, H, n, d]");
    if (t.stride(3) != 1 && t.size(3) != 1) refuse(what, "the channels of a head must be contiguous");
    Heads h;
    h.ptr = t.data_ptr();
    h.device = t.device();
    for (int i = 0; i < 4; ++i) {
        h.size[i] = t.size(i);
        if (h.size[i] >= (1LL << 31)) refuse(what, "a dimension of 2^31 or more");
        if (i < 3) h.stride[i] = h.size[i] == 1 ? 0 : t.stride(i);
    }
    return h;
}

int32_t *int32_of(const at::Tensor &t, std::initializer_list<int64_t> shape, c10::Device device, const char *what) {
    if (t.scalar_type() != at::kInt || !t.is_contiguous() || t.device() != device ||
        !t.sizes().equals(at::IntArrayRef(shape)))
        refuse(what, "expected a contiguous int32 tensor of the call's sizes on its device");
    return static_cast<int32_t *>(t.data_ptr());
}

int32_t *status_of(const at::Tensor &t, c10::Device device) {
    if (t.scalar_type() != at::kInt || t.numel() < 1 || t.device() != device)
        refuse("dev_status", "expected an int32 tensor on the call's device");
    return static_cast<int32_t *>(t.data_ptr());
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, c10::Device device) {
    return at::detail::empty_cuda(shape, type, device, std::nullopt);
}

// The pairs of a rotation on the host: a numpy array of the right type is read in place of a list.
struct Pairs {
    static constexpr int kMost = 64;  // d / 2 at d = 128; the library refuses more before it reads them
    double freq[kMost];
    int32_t axis[kMost];
    int n = 0, pairing = 0;
};

template <class T, class F>
int64_t read_list(PyObject *o, T *out, char format, const char *what, F value) {
    Py_buffer v;
    if (PyObject_CheckBuffer(o) && PyObject_GetBuffer(o, &v, PyBUF_C_CONTIGUOUS | PyBUF_FORMAT) == 0) {
        const bool fits = v.ndim == 1 && v.itemsize == sizeof(T) && v.format && v.format[0] == format && !v.format[1];
        const int64_t n = v.ndim == 1 ? v.shape[0] : -1;
        if (fits) std::copy_n(static_cast<const T *>(v.buf), std::min<int64_t>(n, Pairs::kMost), out);
        PyBuffer_Release(&v);
        if (fits) return n;
    }
    PyErr_Clear();
    PyObject *seq = PySequence_Fast(o, "");
    if (!seq) {
        PyErr_Clear();
        refuse("rope", what);
    }
    const int64_t n = PySequence_Fast_GET_SIZE(seq);
    for (int64_t i = 0; i < std::min<int64_t>(n, Pairs::kMost); ++i) out[i] = value(PySequence_Fast_GET_ITEM(seq, i));
    Py_DECREF(seq);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        refuse("rope", what);
    }
    return n;
}

Pairs pairs_of(PyObject *rope) {
    if (!PyTuple_Check(rope) || PyTuple_GET_SIZE(rope) != 3) refuse("rope", "expected RopeAxes(inv_freq, pair_axis, pairing)");
    Pairs p;
    const int64_t n = read_list(PyTuple_GET_ITEM(rope, 0), p.freq, 'd', "inv_freq is a list of numbers",
                                [](PyObject *x) { return PyFloat_AsDouble(x); });
    const int64_t m = read_list(PyTuple_GET_ITEM(rope, 1), p.axis, 'i', "pair_axis is a list of whole numbers",
                                [](PyObject *x) {
                                    const long i = PyLong_AsLong(x);
                                    return i == static_cast<int32_t>(i) ? static_cast<int32_t>(i) : -1;  // (-1 is refused)
                                });
    if (n != m || n > 1 << 20) refuse("rope", "inv_freq and pair_axis are two lists of the same length");
    p.n = static_cast<int>(n);
    PyObject *name = PyTuple_GET_ITEM(rope, 2);
    if (PyUnicode_Check(name) && PyUnicode_CompareWithASCIIString(name, "interleaved") == 0) p.pairing = 0;
    else if (PyUnicode_Check(name) && PyUnicode_CompareWithASCIIString(name, "half") == 0) p.pairing = 1;
    else refuse("rope", "pairing is \"interleaved\" or \"half\"");
    return p;
}

struct Positions {
    const int32_t *ptr = nullptr;
    int64_t batch_stride = 0;
    int axes = 0;
};

Positions positions_of(PyObject *o, int64_t B, int64_t n, c10::Device device) {
    const at::Tensor &t = tensor(o, "positions");
    if (t.dim() != 2 && t.dim() != 3) refuse("positions", "expected [n, axes] or [B, n, axes]");
    Positions p;
    const int64_t axes = t.size(t.dim() - 1);
    if (axes < 1 || axes > 1 << 20) refuse("positions", "expected [n, axes] or [B, n, axes]");
    p.axes = static_cast<int>(axes);
    p.ptr = t.dim() == 2 ? int32_of(t, {n, axes}, device, "positions") : int32_of(t, {B, n, axes}, device, "positions");
    p.batch_stride = t.dim() == 2 ? 0 : n * axes;
    return p;
}

// KvPages(k_codes, k_exp, v_codes, v_exp) and a page table.
struct Pool {
    uint8_t *k = nullptr, *v = nullptr;
    int32_t *ke = nullptr, *ve = nullptr;
    const int32_t *table = nullptr;
    int pages = 0, heads = 0, block = 0, d = 0, max_pages = 0;
};

Pool pool_of(PyObject *pages, PyObject *page_table, int64_t B, c10::Device device) {
    if (!PyTuple_Check(pages) || PyTuple_GET_SIZE(pages) != 4)
        refuse("pages", "expected KvPages(k_codes, k_exp, v_codes, v_exp)");
    const at::Tensor &k = tensor(PyTuple_GET_ITEM(pages, 0), "k_codes");
    const at::Tensor &v = tensor(PyTuple_GET_ITEM(pages, 2), "v_codes");
    if (k.dim() != 4) refuse("pages", "expected codes [pages, heads, block, d]");
    for (const at::Tensor *t : {&k, &v})
        if (t->scalar_type() != at::kByte || !t->sizes().equals(k.sizes()) || !t->is_contiguous() || t->device() != device)
            refuse("pages", "codes are contiguous uint8 tensors of one shape on the call's device");
    for (int i = 0; i < 4; ++i)
        if (k.size(i) >= (1LL << 31)) refuse("pages", "a dimension of 2^31 or more");
    Pool p;
    p.ke = int32_of(tensor(PyTuple_GET_ITEM(pages, 1), "k_exp"), {k.size(0), k.size(1)}, device, "k_exp");
    p.ve = int32_of(tensor(PyTuple_GET_ITEM(pages, 3), "v_exp"), {k.size(0), k.size(1)}, device, "v_exp");
    p.k = static_cast<uint8_t *>(k.data_ptr());
    p.v = static_cast<uint8_t *>(v.data_ptr());
    p.pages = static_cast<int>(k.size(0));
    p.heads = static_cast<int>(k.size(1));
    p.block = static_cast<int>(k.size(2));
    p.d = static_cast<int>(k.size(3));
    const at::Tensor &t = tensor(page_table, "page_table");
    if (t.dim() != 2 || t.size(1) >= (1LL << 31)) refuse("page_table", "expected int32 [B, max_pages]");
    p.table = int32_of(t, {B, t.size(1)}, device, "page_table");
    p.max_pages = static_cast<int>(t.size(1));
    return p;
}

fvattn_stream_t current_stream(c10::Device device) {
    return reinterpret_cast<fvattn_stream_t>(c10::cuda::getCurrentCUDAStream(device.index()).stream());
}

// The call's own checks and C++ errors as Python's; `n` is the number of arguments wanted.
template <class F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t n, F f) {
    HANDLE_TH_ERRORS
    if (got != n) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return f();
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// rope(Q, K or None, positions, rope, inverse, out_q or None, out_k or None)
// -> (Q, K or None), or the library's status
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject * {
        const Heads q = heads_of(tensor(a[0], "Q"), "Q");
        const bool has_k = a[1] != Py_None;
        Heads k;
        if (has_k) {
            k = heads_of(tensor(a[1], "K"), "K");
            if (k.size[0] != q.size[0] || k.size[2] != q.size[2] || k.size[3] != q.size[3] || k.device != q.device)
                refuse("K", "must match Q in all but its heads");
        } else if (a[6] != Py_None) {
            refuse("out_k", "given without K");
        }
        const Positions pos = positions_of(a[2], q.size[0], q.size[2], q.device);
        const Pairs p = pairs_of(a[3]);
        const int inverse = PyObject_IsTrue(a[4]);
        if (inverse < 0) return nullptr;
        const c10::cuda::CUDAGuard guard(q.device);
        auto out = [&](PyObject *given, const Heads &like, const char *what) {
            at::Tensor t = given != Py_None ? tensor(given, what)
                                            : empty({like.size[0], like.size[1], like.size[2], like.size[3]}, at::kBFloat16,
                                                    like.device);
            if (!heads_of(t, what).like(like)) refuse(what, "wrong shape or device");
            return t;
        };
        const at::Tensor oq = out(a[5], q, "out_q");
        const Heads qo = heads_of(oq, "out_q");
        at::Tensor ok;
        Heads ko;
        if (has_k) {
            ok = out(a[6], k, "out_k");
            ko = heads_of(ok, "out_k");
        }
        const int rc = fvattn_rope(q.ptr, q.stride, const_cast<void *>(qo.ptr), qo.stride, static_cast<int>(q.size[1]), k.ptr,
                                   k.stride, const_cast<void *>(ko.ptr), ko.stride, static_cast<int>(k.size[1]),
                                   static_cast<int>(q.size[0]), static_cast<int>(q.size[2]), static_cast<int>(q.size[3]),
                                   pos.ptr, pos.batch_stride, p.freq, p.axis, p.n, pos.axes, p.pairing, inverse,
                                   current_stream(q.device));
        if (rc != FVATTN_OK) return PyLong_FromLong(rc);
        PyObject *r = PyTuple_New(2);
        if (!r) return nullptr;
        PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(oq));
        PyTuple_SET_ITEM(r, 1, has_k ? THPVariable_Wrap(ok) : Py_NewRef(Py_None));
        return r;
    });
}

// cache_append(K, V, pages, page_table, start, new_lens or None, positions or None, rope or None,
//              dev_status or None) -> dev_status, or the library's status
PyObject *cache_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject * {
        const Heads k = heads_of(tensor(a[0], "K"), "K"), v = heads_of(tensor(a[1], "V"), "V");
        if (!v.like(k)) refuse("V", "must match K");
        const int64_t B = k.size[0];
        const Pool pool = pool_of(a[2], a[3], B, k.device);
        if (pool.heads != k.size[1] || pool.d != k.size[3]) refuse("pages", "heads and d must match K");
        const int32_t *start = int32_of(tensor(a[4], "start"), {B}, k.device, "start");
        const int32_t *new_lens = a[5] == Py_None ? nullptr : int32_of(tensor(a[5], "new_lens"), {B}, k.device, "new_lens");
        if ((a[6] == Py_None) != (a[7] == Py_None)) refuse("positions", "positions and rope belong together");
        Positions pos;
        Pairs p;
        if (a[6] != Py_None) {
            pos = positions_of(a[6], B, k.size[2], k.device);
            p = pairs_of(a[7]);
        }
        const c10::cuda::CUDAGuard guard(k.device);
        const at::Tensor status = a[8] == Py_None ? empty({1}, at::kInt, k.device) : tensor(a[8], "dev_status");
        const int rc = fvattn_cache_append(k.ptr, k.stride, v.ptr, v.stride, static_cast<int>(B), pool.heads,
                                           static_cast<int>(k.size[2]), pool.d, pool.block, pool.k, pool.ke, pool.v,
                                           pool.ve, pool.pages, pool.table, pool.max_pages, start, new_lens, pos.ptr,
                                           pos.batch_stride, p.freq, p.axis, p.n, pos.axes, p.pairing,
                                           status_of(status, k.device), current_stream(k.device));
        return rc != FVATTN_OK ? PyLong_FromLong(rc) : THPVariable_Wrap(status);
    });
}

// cache_attend(Q, pages, page_table, lens, new_lens or None, causal, O or None, LSE or None,
//              workspace or None, dev_status or None) -> (O, LSE, dev_status), or the library's status
PyObject *cache_attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject * {
        const Heads q = heads_of(tensor(a[0], "Q"), "Q");
        const int64_t B = q.size[0], Hq = q.size[1], M = q.size[2];
        const Pool pool = pool_of(a[1], a[2], B, q.device);
        if (pool.heads < 1 || Hq % pool.heads || pool.d != q.size[3])
            refuse("Q", "has a multiple of the cache's heads, and its d");
        const int group = static_cast<int>(Hq / pool.heads);
        const int32_t *lens = int32_of(tensor(a[3], "lens"), {B}, q.device, "lens");
        const int32_t *new_lens = a[4] == Py_None ? nullptr : int32_of(tensor(a[4], "new_lens"), {B}, q.device, "new_lens");
        const int causal = PyObject_IsTrue(a[5]);
        if (causal < 0) return nullptr;
        const c10::cuda::CUDAGuard guard(q.device);
        const at::Tensor O = a[6] == Py_None ? empty({B, Hq, M, q.size[3]}, at::kBFloat16, q.device) : tensor(a[6], "O");
        const Heads o = heads_of(O, "O");
        if (!o.like(q)) refuse("O", "must match Q");
        const at::Tensor LSE = a[7] == Py_None ? empty({B, Hq, M}, at::kFloat, q.device) : tensor(a[7], "LSE");
        if (LSE.scalar_type() != at::kFloat || !LSE.is_contiguous() || LSE.device() != q.device ||
            !LSE.sizes().equals(at::IntArrayRef({B, Hq, M})))
            refuse("LSE", "expected contiguous fp32 [B, H, M]");
        const at::Tensor status = a[9] == Py_None ? empty({1}, at::kInt, q.device) : tensor(a[9], "dev_status");
        at::Tensor ws;
        if (a[8] == Py_None) {
            const size_t need = fvattn_cache_attend_workspace_bytes(static_cast<int>(B), pool.heads, group,
                                                                    static_cast<int>(M), pool.d, pool.block, pool.max_pages);
            ws = empty({static_cast<int64_t>(need > 16 ? need : 16)}, at::kByte, q.device);
        } else {
            ws = tensor(a[8], "workspace");
            if (!ws.is_contiguous() || ws.device() != q.device) refuse("workspace", "expected a contiguous tensor on Q's device");
        }
        const int rc = fvattn_cache_attend(q.ptr, q.stride, static_cast<int>(B), pool.heads, group, static_cast<int>(M), pool.d,
                                           pool.block, pool.k, pool.ke, pool.v, pool.ve, pool.pages, pool.table,
                                           pool.max_pages, lens, new_lens, causal, const_cast<void *>(o.ptr), o.stride,
                                           static_cast<float *>(LSE.data_ptr()), ws.data_ptr(),
                                           static_cast<size_t>(ws.numel() * ws.element_size()),
                                           status_of(status, q.device), current_stream(q.device));
        if (rc != FVATTN_OK) return PyLong_FromLong(rc);
        PyObject *r = PyTuple_New(3);
        if (!r) return nullptr;
        PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(O));
        PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(LSE));
        PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(status));
        return r;
    });
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<rope>("rope"), method<cache_append>("cache_append"),
                         method<cache_attend>("cache_attend"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Calls of libfvattn.so on torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", FVATTN_BUILT_FOR) < 0) Py_CLEAR(m);
    return m;
}
