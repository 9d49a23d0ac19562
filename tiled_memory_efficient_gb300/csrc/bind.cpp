// bind.cpp -- Python binding of the sliding-window, cache and rotary calls (include/attn.h,
// kvcache.h, rope.h): argument checks, output and workspace tensors, the current stream.
//
// A decoding step's kernels take a few microseconds, less than the same checks
// and allocations take in Python (append: 10.9 us of host time a call there, 3.8 us
// of it the C call; attention 26.6 us, 5.9 us of it), so this side is compiled.  It
// holds no computation.  Every function returns None-like results on success,
// a status code (int > 0) from the C call, or -1 for arguments that do not fit
// together, which _lib.py then looks at again to say why.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <optional>
#include <set>
#include <vector>

#include "../../include/attn.h"
#include "../../include/kvcache.h"
#include "../../include/rope.h"

namespace {

// The C entry points, by address (init): this module does not link the library.
struct Fns {
    decltype(&kv8_append_step) append;
    decltype(&kv8_attn_step) attn;
    decltype(&kv8_attn_workspace_size) attn_size;
    decltype(&kv8_copy_pages) copy;
    decltype(&kvp_reserve_step) reserve;
    decltype(&kvp_reassign) reassign;
    decltype(&kvp_compact) compact;
    decltype(&kvp_workspace_size) page_size;
    decltype(&attn_fwd_window) fwd;
    decltype(&attn_fwd_window_workspace_size) fwd_size;
    decltype(&attn_bwd_window) bwd;
    decltype(&attn_bwd_window_workspace_size) bwd_size;
    decltype(&rope_apply) rope;
    decltype(&kv8_append_rope) append_rope;
    decltype(&kv8_attn_shared) attn_shared;
    decltype(&kv8_attn_shared_workspace_size) attn_shared_size;
    decltype(&kvp_find_shared) find_shared;
    decltype(&kvp_plan_words) plan_words;
} fn;

using at::Tensor;

constexpr int kMisfit = -1;

// The tensor behind an argument; an undefined one for None or anything else.
Tensor tensor(PyObject* o) { return THPVariable_Check(o) ? THPVariable_Unpack(o) : Tensor(); }

// CUDA device of a tensor, -1 for another kind or none.
int64_t cuda_of(const Tensor& t) { return t.defined() && t.is_cuda() ? t.get_device() : -1; }

bool fits(const Tensor& t, int64_t dev, at::ScalarType type, at::IntArrayRef shape) {
    return t.defined() && t.is_cuda() && t.get_device() == dev && t.scalar_type() == type &&
           t.sizes() == shape && t.is_contiguous();
}

bool half(const Tensor& t) {
    return t.scalar_type() == at::kHalf || t.scalar_type() == at::kBFloat16;
}
int code(const Tensor& t) { return t.scalar_type() == at::kBFloat16 ? ATTN_BF16 : ATTN_F16; }

// A 32-bit count (larger ones mean "all" to the C calls); false: no integer.
bool count(PyObject* o, int* out) {
    int overflow = 0;
    const long long v = PyLong_AsLongLongAndOverflow(o, &overflow);
    if (v == -1 && !overflow && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    *out = overflow > 0 || v > 0x7fffffff ? 0x7fffffff
           : overflow < 0 || v < -0x7fffffff ? -0x7fffffff
                                             : static_cast<int>(v);
    return true;
}

// An integer that 32 bits hold.
bool whole(PyObject* o, int* out) {
    int overflow = 0;
    const long long v = PyLong_AsLongLongAndOverflow(o, &overflow);
    if (v == -1 && !overflow && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    *out = static_cast<int>(v);
    return !overflow && v == *out;
}

// The softmax scale: None is 1/sqrt(D).
bool scale_of(PyObject* o, int64_t D, float* out) {
    if (o == Py_None) {
        *out = static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
        return true;
    }
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    *out = static_cast<float>(v);
    return true;
}

Tensor empty(at::IntArrayRef shape, at::ScalarType type, int64_t dev) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(
                                at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev))));
}

// An optional tensor argument: the given one after a look at it, or a new one.
bool given_or_new(PyObject* o, Tensor* out, at::IntArrayRef shape, at::ScalarType type, int64_t dev) {
    if (o == Py_None) {
        *out = empty(shape, type, dev);
        return true;
    }
    *out = tensor(o);
    return fits(*out, dev, type, shape);
}

// The same for a workspace (size 0: none is needed).
bool workspace(PyObject* o, Tensor* out, size_t size, int64_t dev) {
    if (o == Py_None) {
        if (size > 0) *out = empty({static_cast<int64_t>(size)}, at::kByte, dev);
        return true;
    }
    *out = tensor(o);
    return cuda_of(*out) == dev && out->is_contiguous();
}
void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
template <typename T>
T* as(const Tensor& t) { return static_cast<T*>(ptr(t)); }
size_t bytes(const Tensor& t) { return t.defined() ? t.nbytes() : 0; }

void* stream_of(int64_t dev) {
    return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
}

// The C calls run without the interpreter's lock: a launch waits when the device's queue
// is full.
struct Unlock {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlock() { PyEval_RestoreThread(state); }
};
template <typename F>
int unlocked(F&& f) {
    const Unlock here;
    return f();
}

// The pools of a cache: [n_pages, Hkv, page, D], or with a leading layer dimension.
struct Pools {
    Tensor k, v, ks, vs;
    int64_t dev = -1, layers = 1, n_pages = 0, heads = 0, page = 0, D = 0;
    bool read(PyObject* const* a, bool with_layers) {
        k = tensor(a[0]), v = tensor(a[1]), ks = tensor(a[2]), vs = tensor(a[3]);
        dev = cuda_of(k);
        if (dev < 0) return false;
        const int64_t d = k.dim();
        if (d != 4 && !(with_layers && d == 5)) return false;
        const auto type = k.scalar_type();
        if (type != at::kFloat8_e4m3fn && type != at::kByte && type != at::kChar) return false;
        const at::IntArrayRef shape = k.sizes();
        if (!k.is_contiguous() || !fits(v, dev, type, shape) ||
            !fits(ks, dev, at::kFloat, shape.slice(0, d - 2)) ||
            !fits(vs, dev, at::kFloat, shape.slice(0, d - 2)))
            return false;
        layers = d == 5 ? shape[0] : 1;
        n_pages = shape[d - 4], heads = shape[d - 3], page = shape[d - 2], D = shape[d - 1];
        return n_pages < (1ll << 31) && heads < (1ll << 31);
    }
};

bool ints(const Tensor& t, int64_t dev, at::IntArrayRef shape) { return fits(t, dev, at::kInt, shape); }
bool int_list(const Tensor& t, int64_t dev, int64_t least) {
    return cuda_of(t) == dev && t.scalar_type() == at::kInt && t.is_contiguous() && t.numel() >= least;
}
bool small(at::IntArrayRef shape) {
    for (const int64_t n : shape)
        if (n >= (1ll << 31)) return false;
    return true;
}

#define MISFIT() return PyLong_FromLong(kMisfit)

// An optional device word: undefined for None.
bool word(PyObject* o, Tensor* out, int64_t dev) {
    if (o == Py_None) return true;
    *out = tensor(o);
    return ints(*out, dev, {1});
}

// What both appends take: (k, v, k_pages, v_pages, k_scale, v_scale, table, lens, n_new | None,
// granted | None).
struct Append {
    Pools p;
    Tensor k, v, table, lens, n_new, granted;
    int64_t B = 0, T = 0, st[3] = {};
    bool read(PyObject* const* a) {
        k = tensor(a[0]), v = tensor(a[1]), table = tensor(a[6]), lens = tensor(a[7]);
        if (!p.read(a + 2, false)) return false;
        if (cuda_of(k) != p.dev || cuda_of(v) != p.dev || k.dim() != 4 || !half(k) ||
            v.scalar_type() != k.scalar_type() || v.sizes() != k.sizes() || !small(k.sizes()))
            return false;
        B = k.size(0), T = k.size(2);
        if (k.size(1) != p.heads || k.size(3) != p.D) return false;
        for (int i = 0; i < 3; ++i) {   // strides of dimensions of size 1 do not matter
            st[i] = k.size(i) == 1 ? 0 : k.stride(i);
            if (k.size(i) != 1 && v.stride(i) != st[i]) return false;
        }
        if (k.stride(3) != 1 || v.stride(3) != 1) return false;
        if (!table.defined() || table.dim() != 2 || !ints(table, p.dev, {B, table.size(1)}) ||
            !ints(lens, p.dev, {B}))
            return false;
        if (a[8] != Py_None) {
            n_new = tensor(a[8]);
            if (!ints(n_new, p.dev, {B})) return false;
        }
        return word(a[9], &granted, p.dev);
    }
};

// (Append) -> rc
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Append x;
    if (n != 10 || !x.read(a)) MISFIT();
    const Pools& p = x.p;
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(p.dev));
    return PyLong_FromLong(unlocked([&] {
        return fn.append(ptr(x.k), ptr(x.v), ptr(p.k), ptr(p.v), as<float>(p.ks), as<float>(p.vs),
                         as<int>(x.table), as<int>(x.lens), as<int>(x.n_new), as<int>(x.granted), x.B, p.heads,
                         x.T, p.D, p.page, p.n_pages, x.table.size(1), x.st[0], x.st[1], x.st[2], code(x.k),
                         stream_of(p.dev));
    }));
    END_HANDLE_TH_ERRORS
}

// A rotation: its frequencies on a device and what the C calls take beside them.
struct Turns {
    Tensor turns;
    int rot = 0, interleaved = 0;
    float amp = 1.0f;
    // One tuple: (turns, rot, interleaved, amplitude, head dim)
    bool read(PyObject* o, int64_t dev, int64_t D) {
        if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 5) return false;
        PyObject* a[5];
        for (int i = 0; i < 5; ++i) a[i] = PyTuple_GET_ITEM(o, i);
        turns = tensor(a[0]);
        int dim;
        if (!whole(a[1], &rot) || !whole(a[2], &interleaved) || a[3] == Py_None || !scale_of(a[3], 1, &amp) ||
            !whole(a[4], &dim))
            return false;
        return dim == D && rot > 0 && fits(turns, dev, at::kLong, {rot / 2});
    }
    const unsigned long long* at() const { return as<unsigned long long>(turns); }
};

// Whether the C calls can read rows where they lie; strides of dimensions of size 1 do not matter.
bool in_place(const Tensor& t) {
    if (t.stride(3) != 1 || reinterpret_cast<uintptr_t>(t.data_ptr()) % 16) return false;
    for (int i = 0; i < 3; ++i)
        if (t.size(i) != 1 && t.stride(i) % 8) return false;
    return true;
}
void strides_of(const Tensor& t, long long* st) {
    for (int i = 0; i < 3; ++i) st[i] = t.size(i) == 1 ? 0 : t.stride(i);
}
Tensor readable(const Tensor& t) { return in_place(t) ? t : t.clone(at::MemoryFormat::Contiguous); }

// Whether a graph follows a tensor, or a forward-mode derivative does.
bool followed(const Tensor& t) {
    return (at::GradMode::is_enabled() && t.requires_grad()) || t._fw_grad(0).defined();
}

// A given result for `like`: rows that no two elements share, of a tensor that no graph follows.
bool result_for(const Tensor& out, const Tensor& like) {
    if (!like.defined() || cuda_of(out) != cuda_of(like) || out.scalar_type() != like.scalar_type() ||
        out.sizes() != like.sizes() || !in_place(out))
        return false;
    // dimension by dimension, the nearest first: each steps over all that the ones before it reach
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int a, int b) { return out.stride(a) < out.stride(b); });
    int64_t reach = out.size(3);
    for (int i : order) {
        if (out.size(i) == 1) continue;
        if (out.stride(i) < reach) return false;
        reach += (out.size(i) - 1) * out.stride(i);
    }
    return !followed(out) && !followed(like);
}
// Two tensors that begin at the same place: a result is not to be another operand.
bool same_place(const Tensor& a, const Tensor& b) {
    return a.defined() && b.defined() && a.data_ptr() == b.data_ptr();
}
// A given result was written to: its version is counted on, as any call that writes to it does.
void written(const Tensor& out) {
    if (!out.is_inference()) out.unsafeGetTensorImpl()->bump_version();
}

// (Append, Turns, q | None, q_out | None) -> q_out, None or rc
PyObject* py_append_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Append x;
    Turns r;
    if (n != 13 || !x.read(a) || !r.read(a[10], x.p.dev, x.p.D)) MISFIT();
    const Pools& p = x.p;
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(p.dev));
    long long st[9] = {x.st[0], x.st[1], x.st[2]};
    Tensor q, out;
    if (a[11] != Py_None) {
        q = tensor(a[11]);
        if (cuda_of(q) != p.dev || q.dim() != 4 || q.scalar_type() != x.k.scalar_type() || q.size(0) != x.B ||
            q.size(2) != x.T || q.size(3) != p.D || !small(q.sizes()))
            MISFIT();
        if (a[12] == Py_None) {
            if (followed(q)) MISFIT();   // (the turned queries would lead nowhere)
            q = readable(q);
            out = empty(q.sizes(), q.scalar_type(), p.dev);
        } else {
            out = tensor(a[12]);
            if (!result_for(out, q) || same_place(out, x.k) || same_place(out, x.v)) MISFIT();
            if (out.data_ptr() != q.data_ptr()) q = readable(q);
        }
        strides_of(q, st + 3);
        strides_of(out, st + 6);
    } else if (a[12] != Py_None) {
        MISFIT();
    }
    const int rc = unlocked([&] {
        return fn.append_rope(ptr(x.k), ptr(x.v), ptr(p.k), ptr(p.v), as<float>(p.ks), as<float>(p.vs),
                              as<int>(x.table), as<int>(x.lens), as<int>(x.n_new), as<int>(x.granted), ptr(q),
                              ptr(out), r.at(), r.rot, r.interleaved, r.amp, x.B, q.defined() ? q.size(1) : 0,
                              p.heads, x.T, p.D, p.page, p.n_pages, x.table.size(1), st, code(x.k),
                              stream_of(p.dev));
    });
    if (rc != ATTN_OK) return PyLong_FromLong(rc);
    if (!out.defined()) Py_RETURN_NONE;
    if (a[12] != Py_None) written(out);
    return THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// Wraps two results.
PyObject* pair(const Tensor& a, const Tensor& b) {
    PyObject* x = THPVariable_Wrap(a);
    PyObject* y = THPVariable_Wrap(b);
    PyObject* r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
}

// What both attentions take: (q, k_pages, v_pages, k_scale, v_scale, table, lens, scale | None), and
// elsewhere n_new | None, granted | None.
struct CacheAttn {
    Pools p;
    Tensor q, table, lens, n_new, granted, out, lse, ws;
    int64_t B = 0, Hq = 0, Nq = 0;
    float scale = 0.0f;
    bool read(PyObject* const* a, PyObject* counts, PyObject* grant) {
        q = tensor(a[0]), table = tensor(a[5]), lens = tensor(a[6]);
        if (!p.read(a + 1, false) || !scale_of(a[7], p.D, &scale)) return false;
        if (cuda_of(q) != p.dev || q.dim() != 4 || !half(q) || q.size(3) != p.D ||
            !q.is_contiguous() || !small(q.sizes()))
            return false;
        B = q.size(0), Hq = q.size(1), Nq = q.size(2);
        if (!table.defined() || table.dim() != 2 || !ints(table, p.dev, {B, table.size(1)}) ||
            !ints(lens, p.dev, {B}))
            return false;
        if (counts != Py_None) {
            n_new = tensor(counts);
            if (!ints(n_new, p.dev, {B})) return false;
        }
        return word(grant, &granted, p.dev);
    }
    // (out | None, lse | None, workspace | None), the last of `size` bytes
    bool results(PyObject* const* a, size_t size) {
        return given_or_new(a[0], &out, q.sizes(), q.scalar_type(), p.dev) &&
               given_or_new(a[1], &lse, {B, Hq, Nq}, at::kFloat, p.dev) &&
               workspace(a[2], &ws, size > 0 ? size : 16, p.dev);
    }
};

// (q, k_pages, v_pages, k_scale, v_scale, table, lens, scale | None, window, sinks,
//  out | None, lse | None, workspace | None, n_new | None, granted | None) -> (out, lse) or rc
PyObject* py_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    CacheAttn x;
    int window, sinks;
    if (n != 15 || !count(a[8], &window) || !count(a[9], &sinks) || !x.read(a, a[13], a[14])) MISFIT();
    const Pools& p = x.p;
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(p.dev));
    if (!x.results(a + 10, fn.attn_size(x.B, x.Hq, p.heads, x.Nq, p.D))) MISFIT();
    const int rc = unlocked([&] {
        return fn.attn(ptr(x.q), ptr(p.k), ptr(p.v), as<float>(p.ks), as<float>(p.vs),
                       as<int>(x.table), as<int>(x.lens), as<int>(x.n_new), as<int>(x.granted), ptr(x.out),
                       as<float>(x.lse), ptr(x.ws), bytes(x.ws), x.B, x.Hq, p.heads, x.Nq, p.D, p.page, p.n_pages,
                       x.table.size(1), x.scale, window, sinks, code(x.q), stream_of(p.dev));
    });
    return rc == ATTN_OK ? pair(x.out, x.lse) : PyLong_FromLong(rc);
    END_HANDLE_TH_ERRORS
}

// (q, k_pages, v_pages, k_scale, v_scale, table, lens, scale | None, plan, out | None, lse | None,
//  workspace | None, n_new | None, granted | None) -> (out, lse) or rc
PyObject* py_attn_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    CacheAttn x;
    if (n != 14 || !x.read(a, a[12], a[13])) MISFIT();
    const Pools& p = x.p;
    const Tensor plan = tensor(a[8]);
    if (x.B > 0x7fffffff || !ints(plan, p.dev, {static_cast<int64_t>(fn.plan_words(static_cast<int>(x.B)))})) MISFIT();
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(p.dev));
    if (!x.results(a + 9, fn.attn_shared_size(x.B, x.Hq, p.heads, x.Nq, p.D))) MISFIT();
    const int rc = unlocked([&] {
        return fn.attn_shared(ptr(x.q), ptr(p.k), ptr(p.v), as<float>(p.ks), as<float>(p.vs), as<int>(x.table),
                              as<int>(x.lens), as<int>(x.n_new), as<int>(x.granted), as<int>(plan), ptr(x.out),
                              as<float>(x.lse), ptr(x.ws), bytes(x.ws), x.B, x.Hq, p.heads, x.Nq, p.D, p.page,
                              p.n_pages, x.table.size(1), x.scale, code(x.q), stream_of(p.dev));
    });
    return rc == ATTN_OK ? pair(x.out, x.lse) : PyLong_FromLong(rc);
    END_HANDLE_TH_ERRORS
}

// (table, lens, page, min_saved, plan | None) -> plan or rc
PyObject* py_find_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 5) MISFIT();
    const Tensor table = tensor(a[0]), lens = tensor(a[1]);
    const int64_t dev = cuda_of(table);
    int page, least;
    if (dev < 0 || table.dim() != 2 || !ints(table, dev, table.sizes()) || !small(table.sizes()) ||
        !ints(lens, dev, {table.size(0)}) || !whole(a[2], &page) || !whole(a[3], &least))
        MISFIT();
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    Tensor plan;
    const int B = static_cast<int>(table.size(0));
    if (!given_or_new(a[4], &plan, {static_cast<int64_t>(fn.plan_words(B))}, at::kInt, dev)) MISFIT();
    const int rc = unlocked([&] {
        return fn.find_shared(as<int>(table), as<int>(lens), B, static_cast<int>(table.size(1)), page, least,
                              as<int>(plan), stream_of(dev));
    });
    return rc == ATTN_OK ? THPVariable_Wrap(plan) : PyLong_FromLong(rc);
    END_HANDLE_TH_ERRORS
}

// (k_pages, v_pages, k_scale, v_scale, src, dst, count, max_count | None) -> rc
PyObject* py_copy(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 8) MISFIT();
    Pools p;
    if (!p.read(a, true)) MISFIT();
    const Tensor src = tensor(a[4]), dst = tensor(a[5]), cnt = tensor(a[6]);
    if (!int_list(src, p.dev, 0) || !int_list(dst, p.dev, 0) || cuda_of(cnt) != p.dev ||
        cnt.scalar_type() != at::kInt || cnt.numel() < 1)
        MISFIT();
    const int64_t room = std::min(src.numel(), dst.numel());
    int most = static_cast<int>(std::min<int64_t>(room, 0x7fffffff));
    if (a[7] != Py_None && (!count(a[7], &most) || most > room)) MISFIT();
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(p.dev));
    return PyLong_FromLong(unlocked([&] {
        return fn.copy(ptr(p.k), ptr(p.v), as<float>(p.ks), as<float>(p.vs), as<int>(src), as<int>(dst),
                       as<int>(cnt), most, p.layers, p.heads, p.page, p.D, p.n_pages, stream_of(p.dev));
    }));
    END_HANDLE_TH_ERRORS
}

// The tensors every bookkeeping call takes.
struct Book {
    Tensor table, refs, info, ws;
    int64_t dev = -1, n_seqs = 0, max_pages = 0, n_pages = 0;
    bool read(PyObject* t, PyObject* r, PyObject* i, PyObject* w) {
        table = tensor(t), refs = tensor(r), info = tensor(i);
        dev = cuda_of(table);
        if (dev < 0 || table.dim() != 2 || !refs.defined() || refs.dim() != 1) return false;
        n_seqs = table.size(0), max_pages = table.size(1), n_pages = refs.size(0);
        if (!ints(table, dev, table.sizes()) || !ints(refs, dev, refs.sizes()) ||
            !ints(info, dev, {4}) || !small(table.sizes()) || !small(refs.sizes()))
            return false;
        const size_t size = w == Py_None ? fn.page_size(n_seqs, max_pages, n_pages) : 0;
        return workspace(w, &ws, size > 0 ? size : 16, dev);
    }
};

// (table, lens, refs, n_new, page, info, window, sinks, workspace | None, granted | None) -> rc
PyObject* py_reserve(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 10) MISFIT();
    Book k;
    int page, window, sinks;
    if (!k.read(a[0], a[2], a[5], a[8]) || !count(a[4], &page) || !count(a[6], &window) ||
        !count(a[7], &sinks))
        MISFIT();
    const Tensor lens = tensor(a[1]), n_new = tensor(a[3]);
    Tensor granted;
    if (!ints(lens, k.dev, {k.n_seqs}) || !ints(n_new, k.dev, {k.n_seqs}) || !word(a[9], &granted, k.dev))
        MISFIT();
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(k.dev));
    return PyLong_FromLong(unlocked([&] {
        return fn.reserve(as<int>(k.table), as<int>(lens), as<int>(k.refs), as<int>(n_new), k.n_seqs,
                          k.max_pages, k.n_pages, page, window, sinks, as<int>(k.info), as<int>(granted),
                          ptr(k.ws), bytes(k.ws), stream_of(k.dev));
    }));
    END_HANDLE_TH_ERRORS
}

// (table, lens, refs, parents, page, copy_src, copy_dst, info, workspace | None) -> rc
PyObject* py_reassign(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 9) MISFIT();
    Book k;
    int page;
    if (!k.read(a[0], a[2], a[7], a[8]) || !count(a[4], &page)) MISFIT();
    const Tensor lens = tensor(a[1]), parents = tensor(a[3]), src = tensor(a[5]), dst = tensor(a[6]);
    if (!ints(lens, k.dev, {k.n_seqs}) || !ints(parents, k.dev, {k.n_seqs}) ||
        !int_list(src, k.dev, k.n_seqs) || !int_list(dst, k.dev, k.n_seqs))
        MISFIT();
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(k.dev));
    return PyLong_FromLong(unlocked([&] {
        return fn.reassign(as<int>(k.table), as<int>(lens), as<int>(k.refs), as<int>(parents),
                           k.n_seqs, k.max_pages, k.n_pages, page, as<int>(src), as<int>(dst),
                           as<int>(k.info), ptr(k.ws), bytes(k.ws), stream_of(k.dev));
    }));
    END_HANDLE_TH_ERRORS
}

// (table, refs, move_src, move_dst, info, table_out, refs_out, workspace | None) -> rc
PyObject* py_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 8) MISFIT();
    Book k;
    if (!k.read(a[0], a[1], a[4], a[7])) MISFIT();
    const Tensor src = tensor(a[2]), dst = tensor(a[3]), to = tensor(a[5]), ro = tensor(a[6]);
    if (!int_list(src, k.dev, k.n_pages / 2) || !int_list(dst, k.dev, k.n_pages / 2) ||
        !ints(to, k.dev, k.table.sizes()) || !ints(ro, k.dev, k.refs.sizes()))
        MISFIT();
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(k.dev));
    return PyLong_FromLong(unlocked([&] {
        return fn.compact(as<int>(k.table), as<int>(k.refs), as<int>(to), as<int>(ro), k.n_seqs,
                          k.max_pages, k.n_pages, as<int>(src), as<int>(dst), as<int>(k.info),
                          ptr(k.ws), bytes(k.ws), stream_of(k.dev));
    }));
    END_HANDLE_TH_ERRORS
}

// q, k, v and the window of a sliding-window call.
struct Window {
    Tensor q, k, v;
    int64_t dev = -1, B = 0, Hq = 0, Hkv = 0, Nq = 0, Nk = 0, D = 0;
    int window = 0, sinks = 0;
    float scale = 0.0f;
    bool read(PyObject* q_, PyObject* k_, PyObject* v_, PyObject* w, PyObject* s, PyObject* sc) {
        return read(tensor(q_), tensor(k_), tensor(v_)) && count(w, &window) && count(s, &sinks) &&
               scale_of(sc, D, &scale);
    }
    bool read(const Tensor& q_, const Tensor& k_, const Tensor& v_) {
        q = q_, k = k_, v = v_;
        dev = cuda_of(q);
        if (dev < 0 || cuda_of(k) != dev || cuda_of(v) != dev || q.dim() != 4 || k.dim() != 4 ||
            !half(q) || k.scalar_type() != q.scalar_type() || v.scalar_type() != q.scalar_type() ||
            v.sizes() != k.sizes() || k.size(0) != q.size(0) || k.size(3) != q.size(3) ||
            !q.is_contiguous() || !k.is_contiguous() || !v.is_contiguous() || !small(q.sizes()) ||
            !small(k.sizes()))
            return false;
        B = q.size(0), Hq = q.size(1), Nq = q.size(2), D = q.size(3), Hkv = k.size(1), Nk = k.size(2);
        return true;
    }
    // Workspace bytes, and the calls themselves.
    size_t fwd_size() const { return fn.fwd_size(B, Hq, Hkv, Nq, Nk, D, window, sinks, code(q)); }
    size_t bwd_size() const { return fn.bwd_size(B, Hq, Hkv, Nq, Nk, D, window, sinks, code(q)); }
    int fwd(const Tensor& out, const Tensor& lse, const Tensor& ws) const {
        return fn.fwd(ptr(q), ptr(k), ptr(v), ptr(out), as<float>(lse), ptr(ws), bytes(ws), B, Hq, Hkv,
                      Nq, Nk, D, scale, window, sinks, code(q), stream_of(dev));
    }
    int bwd(const Tensor& out, const Tensor& dout, const Tensor& lse, const Tensor (&g)[3],
            const Tensor& ws) const {
        return fn.bwd(ptr(q), ptr(k), ptr(v), ptr(out), ptr(dout), as<float>(lse), ptr(g[0]),
                      ptr(g[1]), ptr(g[2]), ptr(ws), bytes(ws), B, Hq, Hkv, Nq, Nk, D, scale, window,
                      sinks, code(q), stream_of(dev));
    }
};

// (q, k, v, window, sinks, scale | None, out | None, lse | None, workspace | None) -> (out, lse) or rc
PyObject* py_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Window w;
    if (n != 9 || !w.read(a[0], a[1], a[2], a[3], a[4], a[5])) MISFIT();
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(w.dev));
    Tensor out, lse, ws;
    if (!given_or_new(a[6], &out, w.q.sizes(), w.q.scalar_type(), w.dev) ||
        !given_or_new(a[7], &lse, {w.B, w.Hq, w.Nq}, at::kFloat, w.dev) ||
        !workspace(a[8], &ws, w.fwd_size(), w.dev))
        MISFIT();
    const int rc = unlocked([&] { return w.fwd(out, lse, ws); });
    return rc == ATTN_OK ? pair(out, lse) : PyLong_FromLong(rc);
    END_HANDLE_TH_ERRORS
}

// (q, k, v, out, dout, lse, window, sinks, scale | None, dq | None, dk | None, dv | None,
//  workspace | None) -> (dq, dk, dv) or rc
PyObject* py_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Window w;
    if (n != 13 || !w.read(a[0], a[1], a[2], a[6], a[7], a[8])) MISFIT();
    const auto type = w.q.scalar_type();
    const Tensor out = tensor(a[3]), dout = tensor(a[4]), lse = tensor(a[5]);
    if (!fits(out, w.dev, type, w.q.sizes()) || !fits(dout, w.dev, type, w.q.sizes()) ||
        !fits(lse, w.dev, at::kFloat, {w.B, w.Hq, w.Nq}))
        MISFIT();
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(w.dev));
    Tensor g[3], ws;
    const size_t size = w.bwd_size();
    for (int i = 0; i < 3; ++i)
        if (!given_or_new(a[9 + i], &g[i], i == 0 ? w.q.sizes() : w.k.sizes(), type, w.dev)) MISFIT();
    if (!workspace(a[12], &ws, size > 0 ? size : 16, w.dev)) MISFIT();
    const int rc = unlocked([&] { return w.bwd(out, dout, lse, g, ws); });
    if (rc != ATTN_OK) return PyLong_FromLong(rc);
    PyObject* r = PyTuple_New(3);
    if (!r) return nullptr;
    for (int i = 0; i < 3; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(g[i]));
    return r;
    END_HANDLE_TH_ERRORS
}

// Refuses a captured backward pass that would hand a gradient to a stream outside the
// capture: the capture would make that stream wait for it, which ends the capture
// and with it the process.  A leaf's gradient is summed on the stream of the first
// live graph that holds the leaf, so a graph recorded outside the capture is enough.
// Looks at the functions above the one being evaluated that the pass will reach;
// called by its backward before it launches anything.
void check_captured_backward() {
    if (c10::cuda::currentStreamCaptureStatusMayInitCtx() == c10::cuda::CaptureStatus::None) return;
    using torch::autograd::Node;
    std::set<const Node*> seen;
    std::vector<std::shared_ptr<Node>> open;
    if (auto node = torch::autograd::get_current_node()) open.push_back(std::move(node));
    while (!open.empty()) {
        const std::shared_ptr<Node> node = std::move(open.back());
        open.pop_back();
        for (uint32_t i = 0; i < node->num_outputs(); ++i) {
            const auto& next = node->next_edge(i).function;
            if (!next || !node->task_should_compute_output(i) || !seen.insert(next.get()).second)
                continue;
            open.push_back(next);
            const auto s = next->stream();
            if (!s || s->device_type() != at::kCUDA ||
                s->id() == c10::cuda::getCurrentCUDAStream(s->device_index()).id())
                continue;
            bool inside = s->id() != 0;   // a branch of this capture?  (0: the default stream)
            if (inside) {
                const c10::cuda::CUDAStreamGuard there(*s);
                inside = c10::cuda::currentStreamCaptureStatusMayInitCtx() !=
                         c10::cuda::CaptureStatus::None;
            }
            TORCH_CHECK(inside, "this backward pass is being captured, but a graph recorded outside the "
                                "capture still holds one of its leaves: drop that graph first");
        }
    }
}

// A call that did not run: a status of the library, or kMisfit.
struct Refused {
    int rc;
};

// Gradients of a pass with create_graph: differentiating them raises.  They would be
// constants to the second pass otherwise, whose result would lack their part.  The node
// that raises leads where the one being evaluated does, so that a pass to any of its
// inputs meets it.
void refuse_second(const Tensor (&g)[3], const Tensor& dout) {
    torch::autograd::edge_list to = torch::autograd::get_current_node()->next_edges();
    to.push_back(torch::autograd::impl::gradient_edge(dout));
    const auto node = std::make_shared<torch::autograd::Error>("window_attention has no second derivative",
                                                               std::move(to));
    for (const Tensor& t : g) torch::autograd::set_history(t, node);
}

// Sliding-window attention as a function of the autograd graph.  (In Python it took 235
// us of host time a training pass: the engine's threads hand the interpreter's lock
// to and fro.)
struct WindowAttention : torch::autograd::Function<WindowAttention> {
    using Context = torch::autograd::AutogradContext;
    static Tensor forward(Context* ctx, const Tensor& q, const Tensor& k, const Tensor& v, int64_t window,
                          int64_t sinks, double scale) {
        Window w;
        if (!w.read(q.contiguous(), k.contiguous(), v.contiguous())) throw Refused{kMisfit};
        w.window = static_cast<int>(window), w.sinks = static_cast<int>(sinks);
        w.scale = static_cast<float>(scale);
        const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(w.dev));
        const Tensor out = empty(w.q.sizes(), w.q.scalar_type(), w.dev);
        const Tensor lse = empty({w.B, w.Hq, w.Nq}, at::kFloat, w.dev);
        Tensor ws;
        if (const size_t size = w.fwd_size()) ws = empty({static_cast<int64_t>(size)}, at::kByte, w.dev);
        if (const int rc = w.fwd(out, lse, ws)) throw Refused{rc};
        ctx->save_for_backward({w.q, w.k, w.v, out, lse});
        ctx->saved_data["window"] = window;
        ctx->saved_data["sinks"] = sinks;
        ctx->saved_data["scale"] = scale;
        return out;
    }
    static torch::autograd::variable_list backward(Context* ctx, torch::autograd::variable_list grads) {
        check_captured_backward();
        const auto saved = ctx->get_saved_variables();
        Window w;
        TORCH_CHECK(w.read(saved[0], saved[1], saved[2]), "attn_bwd_window: the saved tensors changed");
        w.window = static_cast<int>(ctx->saved_data["window"].toInt());
        w.sinks = static_cast<int>(ctx->saved_data["sinks"].toInt());
        w.scale = static_cast<float>(ctx->saved_data["scale"].toDouble());
        const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(w.dev));
        const Tensor dout = grads[0].contiguous();
        const auto type = w.q.scalar_type();
        TORCH_CHECK(fits(dout, w.dev, type, w.q.sizes()) && fits(saved[3], w.dev, type, w.q.sizes()) &&
                        fits(saved[4], w.dev, at::kFloat, {w.B, w.Hq, w.Nq}),
                    "attn_bwd_window: arguments do not fit together");
        const Tensor g[3] = {empty(w.q.sizes(), type, w.dev), empty(w.k.sizes(), type, w.dev),
                             empty(w.k.sizes(), type, w.dev)};
        const Tensor ws = empty({static_cast<int64_t>(std::max<size_t>(w.bwd_size(), 16))}, at::kByte, w.dev);
        const int rc = w.bwd(saved[3], dout, saved[4], g, ws);
        TORCH_CHECK(rc == ATTN_OK, "attn_bwd_window failed with status ", rc);
        if (at::GradMode::is_enabled()) refuse_second(g, grads[0]);   // create_graph
        return {g[0], g[1], g[2], Tensor(), Tensor(), Tensor()};
    }
};

// (q, k, v, window, sinks, scale) -> out or rc; differentiable
PyObject* py_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    int window, sinks;
    float scale;
    const Tensor q = n == 6 ? tensor(a[0]) : Tensor();
    if (!q.defined() || q.dim() != 4 || !count(a[3], &window) || !count(a[4], &sinks) ||
        !scale_of(a[5], q.size(3), &scale))
        MISFIT();
    const Tensor k = tensor(a[1]), v = tensor(a[2]);
    if (!k.defined() || !v.defined()) MISFIT();
    Tensor out;
    const int rc = unlocked([&] {
        try {
            out = WindowAttention::apply(q, k, v, window, sinks, scale);
        } catch (const Refused& r) {
            return r.rc;
        }
        return static_cast<int>(ATTN_OK);
    });
    return rc == ATTN_OK ? THPVariable_Wrap(out) : PyLong_FromLong(rc);
    END_HANDLE_TH_ERRORS
}

// Rotary positions of q and, if there is one, k.
struct RopeCall {
    Tensor q, k, positions;
    Turns r;
    int start = 0, transposed = 0;
    bool read(const Tensor& q_, const Tensor& k_, const Tensor& positions_) {
        q = q_, k = k_, positions = positions_;
        const int64_t dev = cuda_of(q);
        if (dev < 0 || q.dim() != 4 || !half(q) || !small(q.sizes())) return false;
        if (k.defined() && (cuda_of(k) != dev || k.dim() != 4 || k.scalar_type() != q.scalar_type() ||
                            k.size(0) != q.size(0) || k.size(2) != q.size(2) || k.size(3) != q.size(3) ||
                            !small(k.sizes())))
            return false;
        if (positions.defined()) {   // [N], [1, N] or [B, N]
            const int64_t d = positions.dim();
            if (cuda_of(positions) != dev || positions.scalar_type() != at::kInt || (d != 1 && d != 2) ||
                positions.size(d - 1) != q.size(2) || (d == 2 && positions.size(0) != 1 && positions.size(0) != q.size(0)))
                return false;
        }
        return true;
    }
    int64_t dev() const { return q.get_device(); }
    // q_out and k_out are given, or made here: contiguous, as the attention takes them.
    int run(Tensor* q_out, Tensor* k_out) const {
        const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev()));
        const Tensor x = q_out->defined() && q_out->data_ptr() == q.data_ptr() ? q : readable(q);
        const Tensor y = !k.defined() || (k_out->defined() && k_out->data_ptr() == k.data_ptr()) ? k : readable(k);
        if (!q_out->defined()) *q_out = empty(q.sizes(), q.scalar_type(), dev());
        if (k.defined() && !k_out->defined()) *k_out = empty(k.sizes(), k.scalar_type(), dev());
        long long st[14] = {};
        strides_of(x, st);
        strides_of(*q_out, st + 6);
        if (k.defined()) {
            strides_of(y, st + 3);
            strides_of(*k_out, st + 9);
        }
        if (positions.defined()) {
            st[12] = positions.dim() == 2 && positions.size(0) > 1 ? positions.stride(0) : 0;
            st[13] = positions.stride(positions.dim() - 1);
        }
        return fn.rope(ptr(x), ptr(y), ptr(*q_out), ptr(*k_out), r.at(), as<int>(positions), start, x.size(0),
                       x.size(1), k.defined() ? k.size(1) : 0, x.size(2), x.size(3), r.rot, r.interleaved, r.amp,
                       transposed, st, code(x), stream_of(dev()));
    }
};

// The rotation as a function of the autograd graph.  It is linear in its rows: the gradient is
// the transposed rotation of theirs, as a function of the graph again.
struct Rotary : torch::autograd::Function<Rotary> {
    using Context = torch::autograd::AutogradContext;
    using Maybe = std::optional<Tensor>;   // (an argument that is an undefined tensor is an error there)
    static Maybe maybe(const Tensor& t) { return t.defined() ? Maybe(t) : std::nullopt; }
    static torch::autograd::variable_list forward(Context* ctx, const Tensor& q, const Maybe& k_,
                                                  const Maybe& positions_, const Tensor& turns, int64_t start,
                                                  int64_t rot, int64_t interleaved, double amp, int64_t transposed) {
        RopeCall c;
        const Tensor k = k_.value_or(Tensor()), positions = positions_.value_or(Tensor());
        if (!c.read(q, k, positions)) throw Refused{kMisfit};
        c.r.turns = turns, c.r.rot = static_cast<int>(rot), c.r.interleaved = static_cast<int>(interleaved);
        c.r.amp = static_cast<float>(amp);
        c.start = static_cast<int>(start), c.transposed = static_cast<int>(transposed);
        Tensor q_out, k_out;
        if (const int rc = c.run(&q_out, &k_out)) throw Refused{rc};
        ctx->set_materialize_grads(false);
        ctx->save_for_backward({positions, turns});
        ctx->saved_data["start"] = start;
        ctx->saved_data["rot"] = rot;
        ctx->saved_data["interleaved"] = interleaved;
        ctx->saved_data["amp"] = amp;
        ctx->saved_data["transposed"] = transposed;
        if (!k.defined()) return {q_out};
        return {q_out, k_out};
    }
    static torch::autograd::variable_list backward(Context* ctx, torch::autograd::variable_list grads) {
        check_captured_backward();
        const auto saved = ctx->get_saved_variables();
        torch::autograd::variable_list out(9);
        const bool two = grads.size() > 1 && grads[1].defined();
        if (!grads[0].defined() && !two) return out;
        // the first of them that there is takes q's place
        const int first = grads[0].defined() ? 0 : 1;
        try {
            auto g = apply(grads[first], first == 0 && two ? Maybe(grads[1]) : Maybe(), maybe(saved[0]), saved[1],
                           ctx->saved_data["start"].toInt(), ctx->saved_data["rot"].toInt(),
                           ctx->saved_data["interleaved"].toInt(), ctx->saved_data["amp"].toDouble(),
                           1 - ctx->saved_data["transposed"].toInt());
            out[first] = g[0];
            if (g.size() > 1) out[1] = g[1];
        } catch (const Refused& r) {
            TORCH_CHECK(false, "rope_apply failed with status ", r.rc);
        }
        return out;
    }
};

// Wraps q' and, if there is one, k'.
PyObject* rotated(const Tensor& q, const Tensor& k) { return k.defined() ? pair(q, k) : THPVariable_Wrap(q); }

// A forward-mode dual number requires no gradient, and its tangent would be lost: refused, as the other
// differentiable calls refuse it.
void no_tangent(const Tensor& t) {
    TORCH_CHECK_NOT_IMPLEMENTED(!t.defined() || !t._fw_grad(0).defined(),
                                "rotary positions have no forward-mode derivative");
}

// (q, k | None, positions | None, start, Turns) -> q', (q', k') or rc;
// differentiable
PyObject* py_rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    RopeCall c;
    if (n != 5 || (a[1] != Py_None && !tensor(a[1]).defined()) || (a[2] != Py_None && !tensor(a[2]).defined()) ||
        !c.read(tensor(a[0]), tensor(a[1]), tensor(a[2])) || !whole(a[3], &c.start) || !c.r.read(a[4], c.dev(), c.q.size(3)))
        MISFIT();
    no_tangent(c.q);
    no_tangent(c.k);
    Tensor q_out, k_out;
    const bool graph = at::GradMode::is_enabled() &&
                       (c.q.requires_grad() || (c.k.defined() && c.k.requires_grad()));
    const int rc = unlocked([&] {
        if (!graph) return c.run(&q_out, &k_out);
        try {
            auto r = Rotary::apply(c.q, Rotary::maybe(c.k), Rotary::maybe(c.positions), c.r.turns, c.start, c.r.rot,
                                   c.r.interleaved, c.r.amp, 0);
            q_out = r[0];
            if (r.size() > 1) k_out = r[1];
        } catch (const Refused& r) {
            return r.rc;
        }
        return static_cast<int>(ATTN_OK);
    });
    return rc == ATTN_OK ? rotated(q_out, k_out) : PyLong_FromLong(rc);
    END_HANDLE_TH_ERRORS
}

// (q, k | None, positions | None, start, Turns, q_out | None, k_out | None, transposed) -> q', (q', k') or rc
PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    RopeCall c;
    if (n != 8 || (a[1] != Py_None && !tensor(a[1]).defined()) || (a[2] != Py_None && !tensor(a[2]).defined()) ||
        !c.read(tensor(a[0]), tensor(a[1]), tensor(a[2])) || !whole(a[3], &c.start) || !c.r.read(a[4], c.dev(), c.q.size(3)) ||
        !whole(a[7], &c.transposed))
        MISFIT();
    Tensor out[2];
    for (int i = 0; i < 2; ++i) {
        if (a[5 + i] == Py_None) continue;
        const Tensor& like = i == 0 ? c.q : c.k;
        out[i] = tensor(a[5 + i]);
        if (!result_for(out[i], like)) MISFIT();
    }
    if (same_place(out[0], c.k) || same_place(out[1], c.q) || same_place(out[0], out[1])) MISFIT();
    const int rc = unlocked([&] { return c.run(&out[0], &out[1]); });
    for (int i = 0; i < 2 && rc == ATTN_OK; ++i)
        if (a[5 + i] != Py_None) written(out[i]);
    return rc == ATTN_OK ? rotated(out[0], out[1]) : PyLong_FromLong(rc);
    END_HANDLE_TH_ERRORS
}

// (addresses of the C entry points, in Fns' order)
PyObject* py_init(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void* at[sizeof(Fns) / sizeof(void*)];
    if (n != static_cast<Py_ssize_t>(sizeof(at) / sizeof(at[0]))) {
        PyErr_SetString(PyExc_TypeError, "init takes one address per entry point");
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < n; ++i) {
        at[i] = PyLong_AsVoidPtr(a[i]);
        if (!at[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
            return nullptr;
        }
    }
    static_assert(sizeof(at) == sizeof(fn), "one pointer per entry point");
    __builtin_memcpy(&fn, at, sizeof(fn));
    Py_RETURN_NONE;
}

#define METHOD(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD("init", py_init),
                         METHOD("kv8_append", py_append),
                         METHOD("kv8_attn", py_attn),
                         METHOD("kv8_copy_pages", py_copy),
                         METHOD("kvp_reserve", py_reserve),
                         METHOD("kvp_reassign", py_reassign),
                         METHOD("kvp_compact", py_compact),
                         METHOD("attn_fwd_window", py_fwd),
                         METHOD("attn_bwd_window", py_bwd),
                         METHOD("window_attention", py_window),
                         METHOD("rope", py_rope),
                         METHOD("rotary", py_rotary),
                         METHOD("kv8_append_rope", py_append_rope),
                         METHOD("kv8_attn_shared", py_attn_shared),
                         METHOD("kvp_find_shared", py_find_shared),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
