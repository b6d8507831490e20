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
decltype(&kda_paged_attn_sinks) f_attn = nullptr;
decltype(&kda_paged_attn_workspace_size) f_workspace = nullptr;
decltype(&kda_qk_rope) f_rope = nullptr;
decltype(&kda_paged_rope_append) f_rope_append = nullptr;
decltype(&kda_verify_drafts) f_verify = nullptr;
decltype(&kda_verify_drafts_workspace_size) f_verify_ws = nullptr;

constexpr int64_t HEAD = 128;
constexpr int64_t SMALL_RESULTS = 1 << 20;  // bytes: what torch's allocator keeps with other small blocks

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

// The elements of x from `first` on, of the same storage, in a shape of their own (results of
// these calls: nothing to differentiate, so the tensor is made without the dispatcher)
at::Tensor part(const at::Tensor &x, int64_t first, at::IntArrayRef sizes) {
    auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(x.storage()), x.key_set(), x.dtype());
    impl->set_storage_offset(x.storage_offset() + first);
    impl->set_sizes_contiguous(sizes);
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
        at::Tensor pos = part(ints, 0, {T}), cu = part(ints, T, {n + 1}), kv = part(ints, T + n + 1, {n}),
                   head = part(ints, T + 2 * n + 1, {1});
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

// attn(q, k_cache, v_cache, block_table, cu_q, kv_len, max_q, sm_scale, window, k_scale, v_scale, out, lse, workspace, error_word,
// sinks)
PyObject *attn(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject * {
        if (n_args != 16 || !f_attn) throw No();
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
                              (float)a[7].real(), as_int(a[8].integer()), as_int(a[15].integer()), out.data_ptr(), (float *)lse.data_ptr(),
                              ws.data_ptr(), ws.nbytes(), (int32_t *)err, stream_of(dev));
        if (rc != KDA_OK) throw No();
        return tuple_of({&out, &lse});
    });
}

// A [T, heads, 128] tensor of this type on this device whose tokens may lie apart.
struct Rows {
    void *p;
    int64_t T, stride;
    int heads;
};
Rows rows_of(const at::Tensor &x, at::ScalarType t, int device) {
    if (!x.is_cuda() || x.get_device() != device || x.scalar_type() != t || x.dim() != 3 || x.size(2) != HEAD) throw No();
    Rows r{x.data_ptr(), x.size(0), x.size(1) * HEAD, as_int(x.size(1))};
    if (!x.is_contiguous()) {
        if (r.T < 2 || x.stride(2) != 1 || x.stride(1) != HEAD) throw No();
        r.stride = x.stride(0);
    }
    return r;
}
Rows rows_like(const Arg &a, at::Tensor &out, const at::Tensor &x, at::ScalarType t, int device) {
    out = a.none() ? at::empty(x.sizes(), x.options()) : a.tensor();
    if (!out.sizes().equals(x.sizes())) throw No();
    return rows_of(out, t, device);
}
bool truth(const Arg &a) {
    if (a.o != Py_True && a.o != Py_False) throw No();
    return a.o == Py_True;
}
// freq: NULL and 0, or the frequencies and the channels they turn
int turned(const Arg &a, const int64_t *&freq, int &device) {
    freq = nullptr;
    if (a.none()) return 0;
    const at::Tensor &f = given(a, at::kLong, device);
    freq = (const int64_t *)f.data_ptr();
    return as_int(2 * f.numel());
}
// one for each token; none are needed where nothing turns
const int32_t *positions_of(const Arg &a, int rot, int64_t T, int &device) {
    if (a.none() && rot == 0) return nullptr;
    const at::Tensor &x = given(a, at::kInt, device);
    if (x.numel() != T) throw No();
    return (const int32_t *)x.data_ptr();
}

// rope(q, k, positions, freq, amplitude, interleaved, q_weight, k_weight, eps, q_out, k_out)
PyObject *rope(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject * {
        if (n_args != 11 || !f_rope) throw No();
        const Arg *a = reinterpret_cast<const Arg *>(args);
        const at::Tensor &q = a[0].tensor(), &k = a[1].tensor();
        if (!q.is_cuda()) throw No();
        int dev = q.get_device();
        const at::ScalarType t = q.scalar_type();
        const Rows qr = rows_of(q, t, dev), kr = rows_of(k, t, dev);
        if (kr.T != qr.T) throw No();
        const int64_t *freq;
        const int rot = turned(a[3], freq, dev);
        const int32_t *pos = positions_of(a[2], rot, qr.T, dev);
        const float *qw = (const float *)optional(a[6], at::kFloat, dev, HEAD), *kw = (const float *)optional(a[7], at::kFloat, dev, HEAD);
        const c10::cuda::OptionalCUDAGuard guard(q.device());
        at::Tensor qo, ko;
        Rows qor, kor;
        // Small results share an allocation (a token of 16 + 2 heads, its results kept: 15.9 us a call, with two 17.3);
        // who keeps a prompt's keys does not keep its queries' memory too.
        if (a[9].none() && a[10].none() && (q.numel() + k.numel()) * (int64_t)q.element_size() <= SMALL_RESULTS) {
            const at::Tensor buf = at::empty({q.numel() + k.numel()}, q.options());
            qo = part(buf, 0, q.sizes());
            ko = part(buf, q.numel(), k.sizes());
            qor = rows_of(qo, t, dev);
            kor = rows_of(ko, t, dev);
        } else {
            qor = rows_like(a[9], qo, q, t, dev);
            kor = rows_like(a[10], ko, k, t, dev);
        }
        const int rc = f_rope(qr.p, kr.p, pos, freq, (float)a[4].real(), qw, kw, (float)a[8].real(), qr.T,
                              qr.heads, kr.heads, (int)HEAD, rot, truth(a[5]) ? KDA_ROPE_INTERLEAVED : KDA_ROPE_HALF, code_of(t),
                              qr.stride, kr.stride, qor.p, kor.p, qor.stride, kor.stride, stream_of(dev));
        if (rc != KDA_OK) throw No();
        return tuple_of({&qo, &ko});
    });
}

// rope_append(q, k, v, positions, slot_map, freq, k_cache, v_cache, amplitude, interleaved, q_weight, k_weight, eps, k_scale,
// v_scale, q_out, error_word): q_out
PyObject *rope_append(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject * {
        if (n_args != 17 || !f_rope_append) throw No();
        const Arg *a = reinterpret_cast<const Arg *>(args);
        const at::Tensor &q = a[0].tensor();
        if (!q.is_cuda()) throw No();
        int dev = q.get_device();
        const at::ScalarType t = q.scalar_type();
        const Rows qr = rows_of(q, t, dev), kr = rows_of(a[1].tensor(), t, dev), vr = rows_of(a[2].tensor(), t, dev);
        const at::Tensor &slots = given(a[4], at::kLong, dev);
        const Cache c = cache_of(a[6], a[7], dev);
        if (kr.T != qr.T || vr.T != qr.T || kr.heads != c.heads || vr.heads != c.heads || slots.numel() != qr.T) throw No();
        const int64_t *freq;
        const int rot = turned(a[5], freq, dev);
        const int32_t *pos = positions_of(a[3], rot, qr.T, dev);
        const float *qw = (const float *)optional(a[10], at::kFloat, dev, HEAD), *kw = (const float *)optional(a[11], at::kFloat, dev, HEAD);
        const float *ks = scale_of(a[13], c, dev), *vs = scale_of(a[14], c, dev);
        void *err = optional(a[16], at::kInt, dev);
        const c10::cuda::OptionalCUDAGuard guard(q.device());
        at::Tensor qo;
        const Rows qor = rows_like(a[15], qo, q, t, dev);
        const int rc = f_rope_append(qr.p, kr.p, vr.p, pos, (const int64_t *)slots.data_ptr(), freq,
                                     (float)a[8].real(), qw, kw, (float)a[12].real(), qr.T, qr.heads, kr.heads, (int)HEAD, rot,
                                     truth(a[9]) ? KDA_ROPE_INTERLEAVED : KDA_ROPE_HALF, code_of(t), c.code, qr.stride, kr.stride,
                                     vr.stride, qor.p, qor.stride, ks, vs, c.k, c.v, c.pages, c.page_size, c.stride, (int32_t *)err,
                                     stream_of(dev));
        if (rc != KDA_OK) throw No();
        return THPVariable_Wrap(qo);
    });
}

// verify(target, draft_tokens, uniforms, draft, n_draft, workspace, error_word)
PyObject *verify(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject * {
        if (n_args != 7 || !f_verify) throw No();
        const Arg *a = reinterpret_cast<const Arg *>(args);
        const at::Tensor &p = a[0].tensor();
        if (!p.is_cuda() || p.dim() != 3 || p.size(1) < 2) throw No();
        int dev = p.get_device();
        const at::ScalarType t = p.scalar_type();
        const int64_t n = p.size(0), w = p.size(1), v = p.size(2);
        auto rows = [&](const at::Tensor &x, int64_t width, int64_t &seq, int64_t &row) {
            if (!x.is_cuda() || x.get_device() != dev || x.scalar_type() != t || x.dim() != 3 || x.size(0) != n || x.size(1) != width ||
                x.size(2) != v)
                throw No();
            seq = width * v;
            row = v;
            if (!x.is_contiguous()) {
                if (n < 2 || width < 2 || v < 2 || x.stride(2) != 1) throw No();
                seq = x.stride(0);
                row = x.stride(1);
            }
            return x.data_ptr();
        };
        int64_t ts, tr, ds = 0, dr = 0;
        const void *tp = rows(p, w, ts, tr), *dp = a[3].none() ? nullptr : rows(a[3].tensor(), w - 1, ds, dr);
        const at::Tensor &d = given(a[1], at::kInt, dev), &u = given(a[2], at::kFloat, dev);
        if (d.dim() != 2 || d.size(0) != n || d.size(1) != w - 1 || u.dim() != 2 || u.size(0) != n || u.size(1) != w) throw No();
        const int32_t *m = (const int32_t *)optional(a[4], at::kInt, dev, n);
        void *err = optional(a[6], at::kInt, dev);
        const c10::cuda::OptionalCUDAGuard guard(p.device());
        const at::Tensor ints = at::empty({n * (w + 1)}, d.options());
        at::Tensor acc = part(ints, 0, {n}), out = part(ints, n, {n, w}), ws;
        void *work = nullptr;
        size_t bytes = 0;
        if (!a[5].none()) {
            const at::Tensor &given_ws = a[5].tensor();
            if (!given_ws.is_cuda() || !given_ws.is_contiguous() || given_ws.get_device() != dev) throw No();
            work = given_ws.data_ptr();
            bytes = given_ws.nbytes();
        } else if ((bytes = f_verify_ws(as_int(n), as_int(w), as_int(v), code_of(t)))) {
            ws = at::empty({(int64_t)bytes}, d.options().dtype(at::kByte));
            work = ws.data_ptr();
        }
        const int rc = f_verify(tp, dp, (const int32_t *)d.data_ptr(), (const float *)u.data_ptr(), m, as_int(n), as_int(w), as_int(v),
                                code_of(t), ts, tr, ds, dr, (int32_t *)acc.data_ptr(), (int32_t *)out.data_ptr(), work, bytes, (int32_t *)err,
                                stream_of(dev));
        if (rc != KDA_OK) throw No();
        return tuple_of({&acc, &out});
    });
}

// init(tables, append, attn, workspace size, rope, rope_append, verify, workspace size): addresses of the library's functions
PyObject *init(PyObject *, PyObject *const *args, Py_ssize_t n) {
    void *p[8];
    if (n != 8) {
        PyErr_SetString(PyExc_TypeError, "init takes eight addresses");
        return nullptr;
    }
    for (int i = 0; i < 8; ++i) {
        p[i] = PyLong_AsVoidPtr(args[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    f_tables = reinterpret_cast<decltype(f_tables)>(p[0]);
    f_append = reinterpret_cast<decltype(f_append)>(p[1]);
    f_attn = reinterpret_cast<decltype(f_attn)>(p[2]);
    f_workspace = reinterpret_cast<decltype(f_workspace)>(p[3]);
    f_rope = reinterpret_cast<decltype(f_rope)>(p[4]);
    f_rope_append = reinterpret_cast<decltype(f_rope_append)>(p[5]);
    f_verify = reinterpret_cast<decltype(f_verify)>(p[6]);
    f_verify_ws = reinterpret_cast<decltype(f_verify_ws)>(p[7]);
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"init", FAST(init)},     {"tables", FAST(tables)}, {"append", FAST(append)},
                         {"attn", FAST(attn)},     {"rope", FAST(rope)},
                         {"rope_append", FAST(rope_append)},               {"verify", FAST(verify)},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_fast(void) { return PyModule_Create(&module); }
