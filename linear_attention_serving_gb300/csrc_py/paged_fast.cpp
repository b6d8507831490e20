// paged_fast.cpp -- the paged calls' way from Python into the library without the
// interpreter's cost: what paged.py checks and hands over through ctypes in some 15
// microseconds takes two or three here, and the smallest of these calls take less than
// that on the GPU.
//
// Every function looks at its arguments, allocates the outputs, calls the C ABI
// (addresses handed over by `init`) and returns the tensors.  Whatever it does not take
// (another type, a wrong shape, an error of the library) it answers with None: paged.py
// then goes its own way, which says what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "kda.h"

namespace {

decltype(&kda_paged_tables) f_tables = nullptr;
decltype(&kda_paged_append) f_append = nullptr;
decltype(&kda_paged_attn) f_attn = nullptr;
decltype(&kda_paged_attn_workspace_size) f_workspace = nullptr;

constexpr int64_t HEAD = 128;

struct No {};  // not for us: None

struct Arg {
    PyObject *o;
    bool none() const { return o == Py_None; }
    const at::Tensor &tensor() const {
        if (!THPVariable_Check(o)) throw No();
        return THPVariable_Unpack(o);
    }
    int64_t integer() const {
        if (!PyLong_Check(o)) throw No();
        int over = 0;
        const long long v = PyLong_AsLongLongAndOverflow(o, &over);
        if (over || (v == -1 && PyErr_Occurred())) {
            PyErr_Clear();
            throw No();
        }
        return v;
    }
    double real() const {
        if (!PyFloat_Check(o)) throw No();
        return PyFloat_AS_DOUBLE(o);
    }
};

// contiguous, of this type, on this CUDA device (-1: any, returned)
const at::Tensor &given(const Arg &a, at::ScalarType t, int &device) {
    const at::Tensor &x = a.tensor();
    if (!x.is_cuda() || x.scalar_type() != t || !x.is_contiguous()) throw No();
    if (device < 0) device = x.get_device();
    if (x.get_device() != device) throw No();
    return x;
}
void *optional(const Arg &a, at::ScalarType t, int &device, int64_t numel = -1) {
    if (a.none()) return nullptr;
    const at::Tensor &x = given(a, t, device);
    if (numel >= 0 && x.numel() != numel) throw No();
    return x.data_ptr();
}
int as_int(int64_t v) {
    if (v < INT32_MIN || v > INT32_MAX) throw No();
    return (int)v;
}
int code_of(at::ScalarType t) {
    if (t == at::kBFloat16) return KDA_BF16;
    if (t == at::kFloat) return KDA_F32;
    if (t == at::kFloat8_e4m3fn) return KDA_E4M3;
    throw No();
}

struct Cache {
    void *k, *v;
    int code, pages, heads, page_size;
    int64_t stride;
};
// contiguous caches only: pages that lie apart go the other way
Cache cache_of(const Arg &ka, const Arg &va, int &device) {
    const at::Tensor &k = ka.tensor(), &v = va.tensor();
    if (k.dim() != 4 || k.size(3) != HEAD || !v.sizes().equals(k.sizes()) || k.scalar_type() != v.scalar_type()) throw No();
    if (!k.is_cuda() || !v.is_cuda() || k.get_device() != device || v.get_device() != device) throw No();
    Cache c;
    c.stride = k.size(1) * k.size(2) * HEAD;
    if (!(k.is_contiguous() && v.is_contiguous())) {
        if (k.size(0) < 2 || !k.strides().equals(v.strides()) || k.stride(1) != k.size(2) * HEAD || k.stride(2) != HEAD ||
            k.stride(3) != 1)
            throw No();
        c.stride = k.stride(0);
    }
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    c.code = code_of(k.scalar_type());
    c.pages = as_int(k.size(0));
    c.heads = as_int(k.size(1));
    c.page_size = as_int(k.size(2));
    return c;
}
const float *scale_of(const Arg &a, const Cache &c, int &device) {
    if ((c.code == KDA_E4M3) == a.none()) throw No();
    return (const float *)optional(a, at::kFloat, device, c.heads);
}

kda_stream_t stream_of(int device) {
    return (kda_stream_t)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
}

// numel elements of x from `first` on, of the same storage (the integers below: nothing
// to differentiate, so the tensor is made without the dispatcher)
at::Tensor part(const at::Tensor &x, int64_t first, int64_t numel) {
    auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(x.storage()), x.key_set(), x.dtype());
    impl->set_storage_offset(x.storage_offset() + first);
    impl->set_sizes_contiguous({numel});
    return at::Tensor(std::move(impl));
}

PyObject *tuple_of(std::initializer_list<const at::Tensor *> ts) {
    PyObject *r = PyTuple_New((Py_ssize_t)ts.size());
    Py_ssize_t i = 0;
    for (const at::Tensor *t : ts) {
        PyObject *o = r ? THPVariable_Wrap(*t) : nullptr;
        if (!o) {
            Py_XDECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

template <class F> PyObject *guarded(F f) {
    try {
        return f();
    } catch (const No &) {
    } catch (const std::exception &) {  // (an allocation that failed: the other way reports it)
    }
    PyErr_Clear();
    Py_RETURN_NONE;
}

// tables(new_len, ctx_len, block_table, free_pages, free_head, T, page_size, n_pages, error_word)
PyObject *tables(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject * {
        if (n_args != 9 || !f_tables) throw No();
        const Arg *a = reinterpret_cast<const Arg *>(args);
        int dev = -1;
        const at::Tensor &nw = given(a[0], at::kInt, dev), &cx = given(a[1], at::kInt, dev), &tab = given(a[2], at::kInt, dev),
                         &fp = given(a[3], at::kInt, dev), &fh = given(a[4], at::kInt, dev);
        void *err = optional(a[8], at::kInt, dev);
        const int64_t n = nw.numel(), T = a[5].integer();
        if (cx.numel() != n || tab.dim() != 2 || tab.size(0) != n || fh.numel() != 1 || T < 0 || n < 1) throw No();
        const c10::cuda::OptionalCUDAGuard guard(nw.device());
        const auto i32 = nw.options();
        at::Tensor slots = at::empty({T}, i32.dtype(at::kLong)), ints = at::empty({T + 2 * n + 2}, i32);
        at::Tensor pos = part(ints, 0, T), cu = part(ints, T, n + 1), kv = part(ints, T + n + 1, n),
                   head = part(ints, T + 2 * n + 1, 1);
        const int rc = f_tables((const int32_t *)nw.data_ptr(), (const int32_t *)cx.data_ptr(), as_int(n), T,
                                (int32_t *)tab.data_ptr(), as_int(tab.size(1)), (const int32_t *)fp.data_ptr(),
                                as_int(fp.numel()), (const int32_t *)fh.data_ptr(), (int32_t *)head.data_ptr(),
                                as_int(a[6].integer()), as_int(a[7].integer()), (int64_t *)slots.data_ptr(),
                                (int32_t *)pos.data_ptr(), (int32_t *)cu.data_ptr(), (int32_t *)kv.data_ptr(), (int32_t *)err,
                                stream_of(dev));
        if (rc != KDA_OK) throw No();
        return tuple_of({&slots, &pos, &cu, &kv, &head});
    });
}

// append(k, v, slot_map, k_cache, v_cache, k_scale, v_scale, error_word): True when done
PyObject *append(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject * {
        if (n_args != 8 || !f_append) throw No();
        const Arg *a = reinterpret_cast<const Arg *>(args);
        int dev = -1;
        const at::Tensor &k = a[0].tensor();
        const at::Tensor &kk = given(a[0], k.scalar_type(), dev), &v = given(a[1], k.scalar_type(), dev),
                         &slots = given(a[2], at::kLong, dev);
        const Cache c = cache_of(a[3], a[4], dev);
        const float *ks = scale_of(a[5], c, dev), *vs = scale_of(a[6], c, dev);
        void *err = optional(a[7], at::kInt, dev);
        if (kk.dim() != 3 || kk.size(1) != c.heads || kk.size(2) != HEAD || !v.sizes().equals(kk.sizes()) ||
            slots.numel() != kk.size(0))
            throw No();
        const c10::cuda::OptionalCUDAGuard guard(kk.device());
        const int rc = f_append(kk.data_ptr(), v.data_ptr(), (const int64_t *)slots.data_ptr(), kk.size(0), c.heads, (int)HEAD,
                                code_of(kk.scalar_type()), c.code, ks, vs, c.k, c.v, c.pages, c.page_size, c.stride,
                                (int32_t *)err, stream_of(dev));
        if (rc != KDA_OK) throw No();
        Py_RETURN_TRUE;
    });
}

// attn(q, k_cache, v_cache, block_table, cu_q, kv_len, max_q, sm_scale, window, k_scale, v_scale, out, lse, workspace, error_word)
PyObject *attn(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject * {
        if (n_args != 15 || !f_attn) throw No();
        const Arg *a = reinterpret_cast<const Arg *>(args);
        int dev = -1;
        const at::ScalarType t = a[0].tensor().scalar_type();
        const at::Tensor &q = given(a[0], t, dev), &tab = given(a[3], at::kInt, dev), &cu = given(a[4], at::kInt, dev),
                         &kv = given(a[5], at::kInt, dev);
        const Cache c = cache_of(a[1], a[2], dev);
        const float *ks = scale_of(a[9], c, dev), *vs = scale_of(a[10], c, dev);
        void *err = optional(a[14], at::kInt, dev);
        if (q.dim() != 3 || q.size(2) != HEAD) throw No();
        const int64_t T = q.size(0), hq = q.size(1), n = kv.numel();
        if (cu.numel() != n + 1 || tab.dim() != 2 || tab.size(0) != n) throw No();
        const c10::cuda::OptionalCUDAGuard guard(q.device());
        at::Tensor out, lse, ws;
        if (a[11].none()) {
            out = at::empty(q.sizes(), q.options());
        } else {
            out = given(a[11], t, dev);
            if (!out.sizes().equals(q.sizes())) throw No();
        }
        if (a[12].none()) {
            lse = at::empty({T, hq}, q.options().dtype(at::kFloat));
        } else {
            lse = given(a[12], at::kFloat, dev);
            if (lse.dim() != 2 || lse.size(0) != T || lse.size(1) != hq) throw No();
        }
        if (a[13].none()) {
            const size_t need = f_workspace(T, as_int(n), as_int(hq), c.heads);
            if (!need) throw No();
            ws = at::empty({(int64_t)need}, q.options().dtype(at::kByte));
        } else {
            ws = a[13].tensor();
            if (!ws.is_cuda() || !ws.is_contiguous() || ws.get_device() != dev) throw No();
        }
        const int rc = f_attn(q.data_ptr(), c.k, c.v, (const int32_t *)tab.data_ptr(), (const int32_t *)cu.data_ptr(),
                              (const int32_t *)kv.data_ptr(), as_int(n), T, as_int(a[6].integer()), as_int(hq), c.heads,
                              (int)HEAD, code_of(t), c.code, ks, vs, c.pages, c.page_size, c.stride, as_int(tab.size(1)),
                              (float)a[7].real(), as_int(a[8].integer()), out.data_ptr(), (float *)lse.data_ptr(),
                              ws.data_ptr(), ws.nbytes(), (int32_t *)err, stream_of(dev));
        if (rc != KDA_OK) throw No();
        return tuple_of({&out, &lse});
    });
}

// init(tables, append, attn, workspace size): addresses of the library's functions
PyObject *init(PyObject *, PyObject *const *args, Py_ssize_t n) {
    void *p[4];
    if (n != 4) {
        PyErr_SetString(PyExc_TypeError, "init takes four addresses");
        return nullptr;
    }
    for (int i = 0; i < 4; ++i) {
        p[i] = PyLong_AsVoidPtr(args[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    f_tables = reinterpret_cast<decltype(f_tables)>(p[0]);
    f_append = reinterpret_cast<decltype(f_append)>(p[1]);
    f_attn = reinterpret_cast<decltype(f_attn)>(p[2]);
    f_workspace = reinterpret_cast<decltype(f_workspace)>(p[3]);
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"init", FAST(init)},     {"tables", FAST(tables)}, {"append", FAST(append)},
                         {"attn", FAST(attn)},     {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_fast(void) { return PyModule_Create(&module); }
