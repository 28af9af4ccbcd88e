// pa_bind.cpp -- the short way of some Python calls to the C ABI: a module that takes the tensors
// as they are, checks them and calls libpa.so.
//
// A small call's time is its host's: in Python, looking at each tensor's type, device, shape and
// strides and converting some 20 arguments takes 10 to 13 us, more than such a call needs on the
// GPU; here it takes about one.  Each function takes its arguments by position, knows only what a
// call usually gets, and returns None for anything else, which the Python function then takes or
// refuses by name; otherwise what the call returns, or its status as an integer if that is not PA_OK.
// No torch type passes the C ABI: it gets pointers, sizes and the current stream.
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <vector>

#include "pa.h"

namespace {

struct Library {
    decltype(&pa_reshape_and_cache_q8) write_q8 = nullptr;
    decltype(&pa_gather_cache_q8) gather_q8 = nullptr;
    decltype(&pa_decode_q8_workspace_size) decode_q8_size = nullptr;
    decltype(&pa_decode_q8) decode_q8 = nullptr;
    decltype(&pa_prefill_varlen_q8_workspace_size) prefill_q8_size = nullptr;
    decltype(&pa_prefill_varlen_q8) prefill_q8 = nullptr;
    decltype(&pa_qk_norm_mrope) mrope = nullptr;
    decltype(&pa_qk_norm_mrope_cache) mrope_cache = nullptr;
} lib;

using Type = at::ScalarType;

// The call that is being made: the device that its tensors have to be on, whose current stream it
// takes, and whether all its arguments have been as usual.
struct Call {
    int dev;
    bool usual = true;
    Call() : dev((int)c10::cuda::current_device()) {}
    void *stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
    const at::Tensor *tensor(PyObject *o, Type type, int dims) {
        if (!THPVariable_Check(o)) return fail();
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.defined() || !t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || t.dim() != dims ||
            t.layout() != at::kStrided || t.is_conj() || t.is_neg())
            return fail();
        return &t;
    }
    // A contiguous vector of n entries (any number for -1).
    const at::Tensor *vector(PyObject *o, Type type, int64_t n) {
        const at::Tensor *t = tensor(o, type, 1);
        return t && (n < 0 || t->size(0) == n) && t->is_contiguous() ? t : fail();
    }
    // BF16 [tokens, heads, dim] (heads, dim -1: any), each token's heads contiguous; the distance
    // between tokens.
    const at::Tensor *rows(PyObject *o, int64_t tokens, int64_t heads, int64_t dim, int64_t *stride) {
        const at::Tensor *t = tensor(o, Type::BFloat16, 3);
        if (!t || (tokens >= 0 && t->size(0) != tokens) || (heads >= 0 && t->size(1) != heads) ||
            (dim >= 0 && t->size(2) != dim) || t->stride(2) != 1 ||
            (t->size(1) > 1 && t->stride(1) != t->size(2)))
            return fail();
        *stride = t->size(0) > 1 ? t->stride(0) : t->size(1) * t->size(2);
        return t;
    }
    int64_t integer(PyObject *o, int64_t low, int64_t high) {
        if (!PyLong_CheckExact(o)) return fail() ? 0 : 0;
        int over = 0;
        const long long v = PyLong_AsLongLongAndOverflow(o, &over);
        if (over || v < low || v > high) usual = false;
        return v;
    }
    // A list or tuple of ints that fit 32 bits.
    std::vector<int32_t> integers(PyObject *o) {
        std::vector<int32_t> v;
        if (!PyList_CheckExact(o) && !PyTuple_CheckExact(o)) return fail(), v;
        const Py_ssize_t n = PySequence_Fast_GET_SIZE(o);
        PyObject **items = PySequence_Fast_ITEMS(o);
        v.reserve(n + 1);
        for (Py_ssize_t i = 0; i < n; ++i) v.push_back((int32_t)integer(items[i], INT32_MIN, INT32_MAX));
        return v;
    }
    float number(PyObject *o) {
        if (PyFloat_CheckExact(o)) return (float)PyFloat_AS_DOUBLE(o);
        usual = false;
        return 0.f;
    }
    const at::Tensor *fail() {
        usual = false;
        return nullptr;
    }
};

template <typename T = void>
T *ptr(const at::Tensor *t) {
    return static_cast<T *>(t->data_ptr());
}

// What may wait is done without the interpreter's lock, as ctypes and torch do it: a launch waits where the
// stream's queue is full, an allocation perhaps for the GPU, and meanwhile other threads go on, and host
// functions of the stream that take the lock.  Python objects are read before.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// A call of the library.
template <typename R, typename... P, typename... A>
R call(R (*f)(P...), A... args) {
    Unlocked u;
    return f(args...);
}

at::Tensor new_rows(const at::Tensor *like, at::IntArrayRef shape) {
    Unlocked u;
    return at::empty(shape, like->options().dtype(Type::BFloat16).requires_grad(false));
}

// An 8-bit cache of more than one page: what most calls get.
struct CacheQ8 {
    void *k, *v;
    uint8_t *ks, *vs;
    int64_t page_stride, scale_stride, pages;
    int block_size, heads;
    bool read(Call &c, PyObject *const *a) {
        const at::Tensor *kt = c.tensor(a[0], Type::Float8_e4m3fn, 4), *vt = c.tensor(a[1], Type::Float8_e4m3fn, 4);
        const at::Tensor *kst = c.tensor(a[2], Type::Byte, 3), *vst = c.tensor(a[3], Type::Byte, 3);
        if (!c.usual) return false;
        pages = kt->size(0);
        const int64_t bs = kt->size(1), h = kt->size(2), blocks = (bs + PA_Q8_TOKENS - 1) / PA_Q8_TOKENS;
        if (pages < 2 || bs < 1 || bs > 1 << 20 || h < 1 || h > 65535 || kt->size(3) != 256 || kt->stride(3) != 1 ||
            kt->stride(2) != 256 || kt->stride(1) != h * 256 || vt->sizes() != kt->sizes() ||
            vt->strides() != kt->strides() || kst->size(0) != pages || kst->size(1) != blocks || kst->size(2) != h ||
            kst->stride(2) != 1 || kst->stride(1) != h || vst->sizes() != kst->sizes() ||
            vst->strides() != kst->strides())
            return c.fail();
        k = ptr(kt);
        v = ptr(vt);
        ks = ptr<uint8_t>(kst);
        vs = ptr<uint8_t>(vst);
        page_stride = kt->stride(0);
        scale_stride = kst->stride(0);
        block_size = (int)bs;
        heads = (int)h;
        return true;
    }
};

PyObject *none() { Py_RETURN_NONE; }
PyObject *status(int rc) { return PyLong_FromLong(rc); }

template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F f) {
    if (n != want) return none();
    try {
        return f();
    } catch (...) {  // the Python function meets the same and says so
        PyErr_Clear();
        return none();
    }
}

// key, value, the four caches, slot_mapping -> True
PyObject *write_q8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject * {
        Call c;
        CacheQ8 cache;
        int64_t ks, vs;
        if (!cache.read(c, a + 2)) return none();
        const at::Tensor *key = c.rows(a[0], -1, cache.heads, 256, &ks);
        if (!key) return none();
        const int64_t T = key->size(0);
        const at::Tensor *value = c.rows(a[1], T, cache.heads, 256, &vs), *slots = c.vector(a[6], Type::Long, T);
        if (!c.usual || T > 0x7fffffff) return none();
        const int rc = call(lib.write_q8, ptr<pa_bf16>(key), ks, ptr<pa_bf16>(value), vs, cache.k, cache.v, cache.ks,
                            cache.vs, cache.page_stride, cache.scale_stride, cache.pages, ptr<int64_t>(slots), (int)T,
                            cache.heads, 256, cache.block_size, c.stream());
        if (rc) return status(rc);
        Py_RETURN_TRUE;
    });
}

// the four caches, slot_mapping -> (k, v)
PyObject *gather_q8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 5, [&]() -> PyObject * {
        Call c;
        CacheQ8 cache;
        if (!cache.read(c, a)) return none();
        const at::Tensor *slots = c.vector(a[4], Type::Long, -1);
        if (!slots || slots->size(0) > 0x7fffffff) return none();
        const int64_t T = slots->size(0);
        at::Tensor k = new_rows(slots, {T, cache.heads, 256}), v = new_rows(slots, {T, cache.heads, 256});
        const int rc = call(lib.gather_q8, cache.k, cache.v, cache.ks, cache.vs, cache.page_stride,
                            cache.scale_stride, cache.pages, ptr<int64_t>(slots), (int)T, cache.heads, 256,
                            cache.block_size, ptr<pa_bf16>(&k), ptr<pa_bf16>(&v), c.stream());
        if (rc) return status(rc);
        PyObject *kp = THPVariable_Wrap(std::move(k)), *vp = THPVariable_Wrap(std::move(v));
        PyObject *pair = kp && vp ? PyTuple_Pack(2, kp, vp) : nullptr;
        Py_XDECREF(kp);
        Py_XDECREF(vp);
        return pair;
    });
}

// A caller's output like q, or a new one.
bool output(Call &c, PyObject *o, const at::Tensor *q, at::Tensor *out) {
    if (o == Py_None) {
        *out = new_rows(q, q->sizes());
        return true;
    }
    const at::Tensor *t = c.tensor(o, Type::BFloat16, 3);
    if (!t || t->sizes() != q->sizes() || !t->is_contiguous()) return false;
    *out = *t;
    return true;
}

// A caller's workspace, or a new one of need() bytes.
template <typename F>
bool workspace(Call &c, PyObject *o, const at::Tensor *q, at::Tensor *ws, F need) {
    if (o == Py_None) {
        const int64_t bytes = (int64_t)std::max<size_t>(need(), 256);
        Unlocked u;
        *ws = at::empty({bytes}, q->options().dtype(Type::Byte));
        return true;
    }
    if (!THPVariable_Check(o)) return false;
    *ws = THPVariable_Unpack(o);
    return ws->defined() && ws->is_cuda() && ws->get_device() == c.dev && ws->is_contiguous();
}

PyObject *given_or(PyObject *o, at::Tensor &&t) {
    if (o == Py_None) return THPVariable_Wrap(std::move(t));
    Py_INCREF(o);
    return o;
}

// q, the four caches, block_table, seq_lens, scale, max_seq_len, out, workspace -> out
PyObject *decode_q8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject * {
        Call c;
        CacheQ8 cache;
        const at::Tensor *q = c.tensor(a[0], Type::BFloat16, 3);
        if (!q || !q->is_contiguous() || !cache.read(c, a + 1)) return none();
        const int64_t S = q->size(0), hq = q->size(1);
        const at::Tensor *table = c.tensor(a[5], Type::Int, 2), *lens = c.vector(a[6], Type::Int, S);
        const float scale = c.number(a[7]);
        const int64_t most = c.integer(a[8], 1, 0x7fffffff);
        if (!c.usual || q->size(2) != 256 || S < 1 || S > 65535 || hq < 1 || hq > 65535 || table->size(0) < S ||
            table->stride(1) != 1 || table->size(1) * cache.block_size < most)
            return none();
        const int64_t table_stride = table->size(0) > 1 ? table->stride(0) : table->size(1);
        at::Tensor out, ws;
        if (!output(c, a[9], q, &out) || !workspace(c, a[10], q, &ws, [&] {
                return call(lib.decode_q8_size, (int)S, (int)hq, cache.heads, 256, cache.block_size, (int)most);
            }))
            return none();
        const int rc = call(lib.decode_q8, ptr<pa_bf16>(q), cache.k, cache.v, cache.ks, cache.vs, cache.page_stride,
                            cache.scale_stride, cache.pages, ptr<int32_t>(table), table_stride, ptr<int32_t>(lens),
                            (int)S, (int)most, (int)hq, cache.heads, 256, cache.block_size, scale,
                            ptr<pa_bf16>(&out), ptr(&ws), ws.nbytes(), c.stream());
        return rc ? status(rc) : given_or(a[9], std::move(out));
    });
}

// q, the four caches, block_table, cu_seqlens_q, seq_lens_k, causal, scale, out, workspace -> out
PyObject *prefill_q8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject * {
        Call c;
        CacheQ8 cache;
        const at::Tensor *q = c.tensor(a[0], Type::BFloat16, 3);
        if (!q || !q->is_contiguous() || !cache.read(c, a + 1)) return none();
        const at::Tensor *table = c.tensor(a[5], Type::Int, 2);
        const std::vector<int32_t> cu = c.integers(a[6]), lens = c.integers(a[7]);
        const float scale = c.number(a[9]);
        if (!c.usual || !PyBool_Check(a[8]) || lens.empty() || cu.size() != lens.size() + 1 ||
            lens.size() > 0x7fffffff || cu.back() != q->size(0) || q->size(2) != 256 || q->size(1) < 1 ||
            q->size(1) > 65535 || table->size(0) < (int64_t)lens.size() || table->stride(1) != 1 ||
            table->size(1) * cache.block_size < *std::max_element(lens.begin(), lens.end()))
            return none();
        const int64_t table_stride = table->size(0) > 1 ? table->stride(0) : table->size(1);
        const int B = (int)lens.size(), hq = (int)q->size(1), causal = a[8] == Py_True;
        at::Tensor out, ws;
        if (!output(c, a[10], q, &out) || !workspace(c, a[11], q, &ws, [&] {
                return call(lib.prefill_q8_size, cu.data(), lens.data(), B, causal, hq, cache.heads, 256,
                            cache.block_size);
            }))
            return none();
        const int rc = call(lib.prefill_q8, ptr<pa_bf16>(q), cache.k, cache.v, cache.ks, cache.vs, cache.page_stride,
                            cache.scale_stride, cache.pages, ptr<int32_t>(table), table_stride, cu.data(),
                            lens.data(), B, causal, hq, cache.heads, 256, cache.block_size, scale,
                            ptr<pa_bf16>(&out), ptr(&ws), ws.nbytes(), c.stream());
        return rc ? status(rc) : given_or(a[10], std::move(out));
    });
}

// What the rotations with and without a cache have in common.
struct Rope {
    const at::Tensor *q, *k, *qw, *kw, *table, *positions;
    int64_t qs, ks, T, hq, hkv, dim, rot, axes_stride;
    const uint8_t *axes;
    float eps, bias;
    int interleaved, num_axes;
    // q, k, q_weight, k_weight, cos_sin, positions, axes, eps, interleaved, weight_bias
    bool read(Call &c, PyObject *const *a) {
        q = c.rows(a[0], -1, -1, -1, &qs);
        if (!q) return false;
        T = q->size(0);
        hq = q->size(1);
        dim = q->size(2);
        k = c.rows(a[1], T, -1, dim, &ks);
        qw = c.vector(a[2], Type::BFloat16, dim);
        kw = c.vector(a[3], Type::BFloat16, dim);
        table = c.tensor(a[4], Type::Float, 2);
        positions = c.tensor(a[5], Type::Int, 2);
        eps = c.number(a[7]);
        bias = c.number(a[9]);
        if (!c.usual || !PyBytes_CheckExact(a[6]) || !PyBool_Check(a[8])) return c.fail();
        interleaved = a[8] == Py_True;
        hkv = k->size(1);
        rot = table->size(1);
        num_axes = (int)positions->size(0);
        axes = reinterpret_cast<const uint8_t *>(PyBytes_AS_STRING(a[6]));
        axes_stride = positions->size(0) > 1 ? positions->stride(0) : T;
        if (T < 1 || T > 0x7fffffff || hq < 1 || hq > 65535 || hkv < 1 || hkv > 65535 || dim > 256 || rot > 256 ||
            table->size(0) > 0x7fffffff || !table->is_contiguous() || positions->size(1) != T || num_axes < 1 ||
            num_axes > PA_MAX_AXES || positions->stride(1) != 1 || PyBytes_GET_SIZE(a[6]) != rot / 2)
            return c.fail();
        return true;
    }
};

// Rope's, q_out, k_out -> (q, k)
PyObject *mrope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject * {
        Call c;
        Rope r;
        if (!r.read(c, a)) return none();
        at::Tensor q = new_rows(r.q, {r.T, r.hq, r.dim}), k = new_rows(r.q, {r.T, r.hkv, r.dim});
        const int rc =
            call(lib.mrope, ptr<pa_bf16>(r.q), r.qs, ptr<pa_bf16>(r.k), r.ks, ptr<pa_bf16>(r.qw), ptr<pa_bf16>(r.kw),
                 r.bias, r.eps, ptr<float>(r.table), (int)r.table->size(0), (int)r.rot, r.interleaved,
                 ptr<int32_t>(r.positions), r.axes_stride, r.num_axes, r.axes, (int)r.T, (int)r.hq, (int)r.hkv,
                 (int)r.dim, ptr<pa_bf16>(&q), r.hq * r.dim, ptr<pa_bf16>(&k), r.hkv * r.dim, c.stream());
        if (rc) return status(rc);
        PyObject *qp = THPVariable_Wrap(std::move(q)), *kp = THPVariable_Wrap(std::move(k));
        PyObject *pair = qp && kp ? PyTuple_Pack(2, qp, kp) : nullptr;
        Py_XDECREF(qp);
        Py_XDECREF(kp);
        return pair;
    });
}

// Rope's, v, k_cache, v_cache, slot_mapping -> q (BF16 caches)
PyObject *mrope_cache(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 14, [&]() -> PyObject * {
        Call c;
        Rope r;
        int64_t vs;
        if (!r.read(c, a)) return none();
        const at::Tensor *v = c.rows(a[10], r.T, r.hkv, r.dim, &vs), *slots = c.vector(a[13], Type::Long, r.T);
        const at::Tensor *kc = c.tensor(a[11], Type::BFloat16, 4), *vc = c.tensor(a[12], Type::BFloat16, 4);
        if (!c.usual || kc->size(2) != r.hkv || kc->size(3) != r.dim || kc->stride(3) != 1 ||
            kc->stride(2) != r.dim || kc->stride(1) != r.hkv * r.dim || kc->size(1) > 0x7fffffff ||
            vc->sizes() != kc->sizes() || vc->strides() != kc->strides())
            return none();
        at::Tensor q = new_rows(r.q, {r.T, r.hq, r.dim});
        const int rc =
            call(lib.mrope_cache, ptr<pa_bf16>(r.q), r.qs, ptr<pa_bf16>(r.k), r.ks, ptr<pa_bf16>(v), vs,
                 ptr<pa_bf16>(r.qw), ptr<pa_bf16>(r.kw), r.bias, r.eps, ptr<float>(r.table), (int)r.table->size(0),
                 (int)r.rot, r.interleaved, ptr<int32_t>(r.positions), r.axes_stride, r.num_axes, r.axes, (int)r.T,
                 (int)r.hq, (int)r.hkv, (int)r.dim, ptr<pa_bf16>(&q), r.hq * r.dim, (int)PA_CACHE_BF16, ptr(kc),
                 ptr(vc), kc->stride(0), kc->size(0), ptr<int64_t>(slots), (int)kc->size(1), c.stream());
        if (rc) return status(rc);
        return THPVariable_Wrap(std::move(q));
    });
}

// The library's path: looks its calls up.
PyObject *load(PyObject *, PyObject *path) {
    const char *name = PyUnicode_AsUTF8(path);
    if (!name) return nullptr;
    void *h = dlopen(name, RTLD_NOW | RTLD_LOCAL);
    if (!h) {
        PyErr_SetString(PyExc_RuntimeError, dlerror());
        return nullptr;
    }
    bool all = true;
    auto find = [&](auto &f, const char *symbol) {
        f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(h, symbol));
        all = all && f;
    };
    find(lib.write_q8, "pa_reshape_and_cache_q8");
    find(lib.gather_q8, "pa_gather_cache_q8");
    find(lib.decode_q8_size, "pa_decode_q8_workspace_size");
    find(lib.decode_q8, "pa_decode_q8");
    find(lib.prefill_q8_size, "pa_prefill_varlen_q8_workspace_size");
    find(lib.prefill_q8, "pa_prefill_varlen_q8");
    find(lib.mrope, "pa_qk_norm_mrope");
    find(lib.mrope_cache, "pa_qk_norm_mrope_cache");
    if (!all) {
        PyErr_SetString(PyExc_RuntimeError, "the library lacks a call of its header");
        return nullptr;
    }
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"load", load, METH_O, nullptr},
                         {"write_q8", FAST(write_q8)},
                         {"gather_q8", FAST(gather_q8)},
                         {"decode_q8", FAST(decode_q8)},
                         {"prefill_q8", FAST(prefill_q8)},
                         {"mrope", FAST(mrope)},
                         {"mrope_cache", FAST(mrope_cache)},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "pa_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_pa_bind() { return PyModule_Create(&module); }
