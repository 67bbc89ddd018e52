// CPython binding of the rotate-and-append and block-sparse entry points.
//
// A decode step calls these once per layer, and on a small batch the kernels
// take a few microseconds: checking a dozen tensors and marshalling some
// thirty arguments in Python takes longer than they do (14 us against 2 to 8
// on a Grace host).  Here the same checks read the tensors' fields directly.
// The library itself stays a plain C ABI: the addresses of its functions are
// handed over by bind(), so both bindings use one loaded copy.
//
// Each function raises TypeError or ValueError for tensors that do not fit,
// returns the library's status as an int when that is not PA_OK, and None
// otherwise.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "pa.h"

namespace {

decltype(&pa_rope_append) f_rope_append;
decltype(&pa_block_summary) f_block_summary;
decltype(&pa_sparse_select) f_sparse_select;
decltype(&pa_sparse_decode) f_sparse_decode;
decltype(&pa_sparse_attend) f_sparse_attend;

// Thrown after a Python exception has been set.
struct Raised {};

template <class... A>
[[noreturn]] void raise(PyObject *type, const char *fmt, A... a) {
    PyErr_Format(type, fmt, a...);
    throw Raised{};
}

const char *name_of(at::ScalarType t) { return c10::toString(t); }

std::string shape_of(const at::Tensor &t) {
    std::string s = "(";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + ")";
}

// The tensors of one call: all have to be on the current CUDA device.
class Call {
public:
    // A tensor argument, or null for None where `optional`.
    const at::Tensor *get(PyObject *o, const char *name, bool optional = false) {
        if (optional && o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a torch.Tensor", name);
        const at::Tensor &t = THPVariable_Unpack(o);
        if (count_ < kMost) {
            seen_[count_] = &t;
            names_[count_++] = name;
        }
        return &t;
    }
    const at::Tensor *dense(PyObject *o, const char *name, at::ScalarType type, int ndim = -1, bool optional = false) {
        const at::Tensor *t = get(o, name, optional);
        if (!t) return nullptr;
        if (t->scalar_type() != type)
            raise(PyExc_TypeError, "%s has dtype %s; expected %s", name, name_of(t->scalar_type()), name_of(type));
        check_dense(*t, name, ndim);
        return t;
    }
    const at::Tensor *shaped(PyObject *o, const char *name, at::ScalarType type, std::initializer_list<int64_t> shape,
                             bool optional = false) {
        const at::Tensor *t = dense(o, name, type, -1, optional);
        if (t && !(t->sizes() == at::IntArrayRef(shape))) {
            std::string want = "(";
            for (int64_t n : shape) want += (want.size() > 1 ? ", " : "") + std::to_string(n);
            raise(PyExc_ValueError, "%s must have shape %s) (got %s)", name, want.c_str(), shape_of(*t).c_str());
        }
        return t;
    }
    // A cache [blocks, heads, block_size, head_dim] of bf16 or E4M3 codes.
    const at::Tensor *cache(PyObject *o, const char *name, pa_kv_dtype *type) {
        const at::Tensor *t = get(o, name);
        const auto s = t->scalar_type();
        if (s != at::kBFloat16 && s != at::kByte && s != at::kFloat8_e4m3fn)
            raise(PyExc_TypeError, "%s has dtype %s; expected bfloat16, uint8 or float8_e4m3fn", name, name_of(s));
        check_dense(*t, name, 4);
        *type = s == at::kBFloat16 ? PA_KV_BF16 : PA_KV_FP8_E4M3;
        return t;
    }
    // bf16 [tokens, heads, head_dim] whose tokens may be a stride apart.
    const at::Tensor *rows(PyObject *o, const char *name, int64_t *stride, bool optional = false) {
        const at::Tensor *t = get(o, name, optional);
        if (!t) return nullptr;
        if (t->scalar_type() != at::kBFloat16)
            raise(PyExc_TypeError, "%s has dtype %s; expected bfloat16", name, name_of(t->scalar_type()));
        if (t->dim() != 3) raise(PyExc_ValueError, "%s must have 3 dimensions (got shape %s)", name, shape_of(*t).c_str());
        if ((t->size(2) > 1 && t->stride(2) != 1) || (t->size(1) > 1 && t->stride(1) != t->size(2)))
            raise(PyExc_ValueError, "%s: each token's [heads, head_dim] rows must be dense", name);
        *stride = t->size(0) > 1 ? t->stride(0) : t->size(1) * t->size(2);
        return t;
    }
    // The stream to use; last of the checks, the tensors' device.
    cudaStream_t stream(PyObject *o) {
        const c10::Device dev = seen_[0]->device();
        if (!dev.is_cuda()) raise(PyExc_ValueError, "%s must be a CUDA tensor (got %s)", names_[0], dev.str().c_str());
        for (int i = 1; i < count_; ++i)
            if (seen_[i]->device() != dev)
                raise(PyExc_ValueError, "%s is on %s; expected %s: one CUDA tensor like the others", names_[i],
                      seen_[i]->device().str().c_str(), dev.str().c_str());
        const auto now = c10::cuda::current_device();
        if (dev.index() != now)
            raise(PyExc_ValueError, "the tensors are on %s, but the current device is cuda:%d", dev.str().c_str(), static_cast<int>(now));
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream(now).stream();
        PyObject *raw = PyObject_GetAttrString(o, "cuda_stream");
        if (!raw) throw Raised{};
        void *p = PyLong_AsVoidPtr(raw);
        Py_DECREF(raw);
        if (!p && PyErr_Occurred()) throw Raised{};
        return static_cast<cudaStream_t>(p);
    }

private:
    static void check_dense(const at::Tensor &t, const char *name, int ndim) {
        if (!t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
        if (ndim >= 0 && t.dim() != ndim)
            raise(PyExc_ValueError, "%s must have %d dimensions (got shape %s)", name, ndim, shape_of(t).c_str());
    }
    static constexpr int kMost = 16;
    const at::Tensor *seen_[kMost];
    const char *names_[kMost];
    int count_ = 0;
};

template <class T>
T *ptr(const at::Tensor *t) {
    return t ? static_cast<T *>(t->data_ptr()) : nullptr;
}

int to_int(PyObject *o, const char *name) {
    const long x = PyLong_AsLong(o);
    if (x == -1 && PyErr_Occurred()) throw Raised{};
    if (x != static_cast<int>(x)) raise(PyExc_ValueError, "%s is out of range", name);
    return static_cast<int>(x);
}

float to_float(PyObject *o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Raised{};
    return static_cast<float>(x);
}

int size(const at::Tensor *t, int i) {
    const int64_t n = t->size(i);
    if (n > 0x7fffffff) raise(PyExc_ValueError, "a dimension of %lld is out of range", static_cast<long long>(n));
    return static_cast<int>(n);
}

struct Caches {
    const at::Tensor *k, *v, *k_scales, *v_scales;
    pa_kv_dtype type;
    int blocks, heads, block, dim;
    Caches(Call &c, PyObject *kc, PyObject *vc, PyObject *ks, PyObject *vs) {
        pa_kv_dtype vtype;
        k = c.cache(kc, "k_cache", &type);
        v = c.cache(vc, "v_cache", &vtype);
        if (vtype != type || v->sizes() != k->sizes()) raise(PyExc_ValueError, "v_cache must be like k_cache");
        if ((ks == Py_None) != (vs == Py_None))
            raise(PyExc_ValueError, "k_scales and v_scales must both be given or both be None");
        blocks = size(k, 0), heads = size(k, 1), block = size(k, 2), dim = size(k, 3);
        k_scales = c.shaped(ks, "k_scales", at::kFloat, {heads}, true);
        v_scales = c.shaped(vs, "v_scales", at::kFloat, {heads}, true);
    }
};

struct Rows {
    const at::Tensor *q, *tables, *lens;
    int rows, heads, dim, width;
    Rows(Call &c, PyObject *qo, PyObject *to, PyObject *lo) {
        q = c.dense(qo, "q", at::kBFloat16, 3);
        tables = c.dense(to, "block_tables", at::kInt, 2);
        rows = size(q, 0), heads = size(q, 1), dim = size(q, 2), width = size(tables, 1);
        if (tables->size(0) != rows) raise(PyExc_ValueError, "block_tables needs one row per query row");
        lens = c.shaped(lo, "context_lens", at::kInt, {rows});
    }
};

// Python's lock is given up while the library launches: a full launch queue
// makes that wait for the GPU.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// Runs a function of (args) and turns what it throws into Python's errors.
template <class F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, F &&body) {
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
        return nullptr;
    }
    try {
        const pa_status st = body();
        if (st != PA_OK) return PyLong_FromLong(st);
        Py_RETURN_NONE;
    } catch (const Raised &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyObject *rope_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 16, [&] {
        Call c;
        int64_t qs = 0, ks = 0, vs = 0;
        const at::Tensor *k = c.rows(a[1], "k", &ks), *v = c.rows(a[2], "v", &vs);
        const Caches cc(c, a[6], a[7], a[12], a[13]);
        const int T = size(k, 0);
        if (v->sizes() != k->sizes() || k->size(1) != cc.heads || k->size(2) != cc.dim)
            raise(PyExc_ValueError, "inconsistent K/V and cache shapes");
        const at::Tensor *pos = c.dense(a[3], "positions", at::kInt);
        if ((pos->dim() != 1 && pos->dim() != 2) || pos->size(-1) != T)
            raise(PyExc_ValueError, "positions must be [tokens] or [axes, tokens] (got %s)", shape_of(*pos).c_str());
        const at::Tensor *freq = c.dense(a[4], "inv_freq", at::kDouble, 1);
        if (freq->size(0) > 65536) raise(PyExc_ValueError, "inv_freq is longer than half a head");
        const at::Tensor *axis = c.shaped(a[8], "pair_axis", at::kInt, {freq->size(0)}, true);
        const at::Tensor *slots = c.shaped(a[5], "slot_mapping", at::kInt, {T});
        const at::Tensor *q = c.rows(a[0], "q", &qs, true), *out = nullptr;
        if (q) {
            if (q->size(0) != T || q->size(2) != cc.dim) raise(PyExc_ValueError, "inconsistent q and k shapes");
            out = c.shaped(a[14], "out", at::kBFloat16, {T, q->size(1), cc.dim});
        }
        const int adjacent = PyObject_IsTrue(a[9]);
        if (adjacent < 0) throw Raised{};
        const float magnitude = to_float(a[10]), kv_scale = to_float(a[11]);
        const int axes = pos->dim() == 2 ? size(pos, 0) : 1, rotary = 2 * size(freq, 0), heads = q ? size(q, 1) : 0;
        const cudaStream_t s = c.stream(a[15]);
        const Unlocked unlocked;
        return f_rope_append(ptr<void>(q), qs, k->data_ptr(), ks, v->data_ptr(), vs, ptr<int32_t>(pos), axes,
                             ptr<double>(freq), ptr<int32_t>(axis), rotary, adjacent, magnitude, ptr<int32_t>(slots), T, heads,
                             ptr<void>(out), cc.k->data_ptr(),
                             cc.v->data_ptr(), cc.blocks, cc.heads, cc.dim, cc.block, cc.type, kv_scale, ptr<float>(cc.k_scales),
                             ptr<float>(cc.v_scales), s);
    });
}

PyObject *block_summary(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 5, [&] {
        Call c;
        pa_kv_dtype type;
        const at::Tensor *k = c.cache(a[0], "k_cache", &type);
        const at::Tensor *slots = c.dense(a[1], "slot_mapping", at::kInt, 1);
        const at::Tensor *sum = c.shaped(a[2], "summary", at::kChar, {k->size(0), k->size(1), 2, k->size(3)});
        const at::Tensor *ex = c.shaped(a[3], "exponents", at::kChar, {k->size(0), k->size(1)});
        const int T = size(slots, 0), blocks = size(k, 0), heads = size(k, 1), block = size(k, 2), dim = size(k, 3);
        const cudaStream_t s = c.stream(a[4]);
        const Unlocked unlocked;
        return f_block_summary(k->data_ptr(), ptr<int32_t>(slots), T, blocks, heads, dim, block, type, ptr<int8_t>(sum),
                               ptr<int8_t>(ex), s);
    });
}

PyObject *sparse_select(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 12, [&] {
        Call c;
        const Rows r(c, a[0], a[3], a[4]);
        const at::Tensor *sum = c.dense(a[1], "summary", at::kChar, 4);
        const int blocks = size(sum, 0), heads = size(sum, 1), top_k = to_int(a[6], "top_k");
        c.shaped(a[1], "summary", at::kChar, {blocks, heads, 2, r.dim});
        const at::Tensor *ex = c.shaped(a[2], "exponents", at::kChar, {blocks, heads});
        const at::Tensor *sel = c.shaped(a[9], "selected", at::kInt, {r.rows, heads, top_k});
        const at::Tensor *cnt = c.shaped(a[10], "counts", at::kInt, {r.rows, heads});
        const int block = to_int(a[5], "block_size"), sink = to_int(a[7], "sink_blocks"), recent = to_int(a[8], "recent_blocks");
        const cudaStream_t s = c.stream(a[11]);
        const Unlocked unlocked;
        return f_sparse_select(r.q->data_ptr(), ptr<int8_t>(sum), ptr<int8_t>(ex), ptr<int32_t>(r.tables), r.width,
                               ptr<int32_t>(r.lens), r.rows, r.heads, heads, r.dim, blocks, block, top_k, sink, recent,
                               ptr<int32_t>(sel), ptr<int32_t>(cnt), s);
    });
}

PyObject *sparse_decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 14, [&] {
        Call c;
        const Rows r(c, a[0], a[3], a[4]);
        const Caches cc(c, a[1], a[2], a[9], a[10]);
        if (cc.dim != r.dim) raise(PyExc_ValueError, "inconsistent q / cache shapes");
        const at::Tensor *sel = c.dense(a[5], "selected", at::kInt, 3);
        const int top_k = size(sel, 2);
        c.shaped(a[5], "selected", at::kInt, {r.rows, cc.heads, top_k});
        const at::Tensor *cnt = c.shaped(a[6], "counts", at::kInt, {r.rows, cc.heads});
        const at::Tensor *out = c.shaped(a[12], "out", at::kBFloat16, {r.rows, r.heads, r.dim});
        const float softmax_scale = to_float(a[7]), kv_scale = to_float(a[8]);
        const int splits = to_int(a[11], "splits");
        const cudaStream_t s = c.stream(a[13]);
        const Unlocked unlocked;
        return f_sparse_decode(r.q->data_ptr(), cc.k->data_ptr(), cc.v->data_ptr(), ptr<int32_t>(r.tables), r.width,
                               ptr<int32_t>(r.lens), r.rows, r.heads, cc.heads, r.dim, cc.blocks, cc.block, cc.type, kv_scale,
                               ptr<float>(cc.k_scales), ptr<float>(cc.v_scales), softmax_scale, ptr<int32_t>(sel),
                               ptr<int32_t>(cnt), top_k, splits, out->data_ptr(), s);
    });
}

PyObject *sparse_attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 18, [&] {
        Call c;
        const Rows r(c, a[0], a[5], a[6]);
        const Caches cc(c, a[1], a[2], a[12], a[13]);
        if (cc.dim != r.dim) raise(PyExc_ValueError, "inconsistent q / cache shapes");
        const int top_k = to_int(a[7], "top_k");
        const at::Tensor *sum = c.shaped(a[3], "summary", at::kChar, {cc.blocks, cc.heads, 2, r.dim});
        const at::Tensor *ex = c.shaped(a[4], "exponents", at::kChar, {cc.blocks, cc.heads});
        const at::Tensor *sel = c.shaped(a[14], "selected", at::kInt, {r.rows, cc.heads, top_k});
        const at::Tensor *cnt = c.shaped(a[15], "counts", at::kInt, {r.rows, cc.heads});
        const at::Tensor *out = c.shaped(a[16], "out", at::kBFloat16, {r.rows, r.heads, r.dim});
        const int sink = to_int(a[8], "sink_blocks"), recent = to_int(a[9], "recent_blocks");
        const float softmax_scale = to_float(a[10]), kv_scale = to_float(a[11]);
        const cudaStream_t s = c.stream(a[17]);
        const Unlocked unlocked;
        return f_sparse_attend(r.q->data_ptr(), cc.k->data_ptr(), cc.v->data_ptr(), ptr<int8_t>(sum), ptr<int8_t>(ex),
                               ptr<int32_t>(r.tables), r.width, ptr<int32_t>(r.lens), r.rows, r.heads, cc.heads, r.dim, cc.blocks,
                               cc.block, cc.type, kv_scale, ptr<float>(cc.k_scales), ptr<float>(cc.v_scales), softmax_scale, top_k,
                               sink, recent, ptr<int32_t>(sel), ptr<int32_t>(cnt), out->data_ptr(), s);
    });
}

// bind(rope_append, block_summary, sparse_select, sparse_decode, sparse_attend): addresses in the loaded library
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 5, [&] {
        void *p[5];
        for (int i = 0; i < 5; ++i) {
            p[i] = PyLong_AsVoidPtr(a[i]);
            if (!p[i]) {
                if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
                throw Raised{};
            }
        }
        f_rope_append = reinterpret_cast<decltype(f_rope_append)>(p[0]);
        f_block_summary = reinterpret_cast<decltype(f_block_summary)>(p[1]);
        f_sparse_select = reinterpret_cast<decltype(f_sparse_select)>(p[2]);
        f_sparse_decode = reinterpret_cast<decltype(f_sparse_decode)>(p[3]);
        f_sparse_attend = reinterpret_cast<decltype(f_sparse_attend)>(p[4]);
        return PA_OK;
    });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)), METH_FASTCALL
PyMethodDef methods[] = {
    {"bind", FAST(bind), nullptr},
    {"rope_append", FAST(rope_append), nullptr},
    {"block_summary", FAST(block_summary), nullptr},
    {"sparse_select", FAST(sparse_select), nullptr},
    {"sparse_decode", FAST(sparse_decode), nullptr},
    {"sparse_attend", FAST(sparse_attend), nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pa_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pa_binding() { return PyModule_Create(&module); }
