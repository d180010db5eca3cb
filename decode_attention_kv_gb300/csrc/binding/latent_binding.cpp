// latent_binding.cpp -- the latent-cache and serving-step calls of kvd.py, from torch
// tensors to the C entry points: argument checks, outputs, device and stream.  A decode loop
// makes these calls every few microseconds; with the same checks in Python and 18
// to 25 arguments converted by ctypes the host took 9.3 us for an append, 16 for a
// verification, 20 and 26 for the attentions; now 2.8, 5.8, 11 and 13 (their
// outputs' allocation among it).
//
// The entry points come from the library that kvd.py has loaded (bind); errors
// are raised by kvd.py's own check.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <initializer_list>
#include <string>

#include "../../../include/kvd.h"

namespace {

decltype(&kvd_append_latent) g_append = nullptr;
decltype(&kvd_attend_latent_workspace_bytes) g_workspace = nullptr;
decltype(&kvd_attend_latent) g_attend = nullptr;
decltype(&kvd_attend_expanded) g_expanded = nullptr;
decltype(&kvd_verify_drafts) g_verify = nullptr;
decltype(&kvd_plan_pages) g_plan_pages = nullptr;
decltype(&kvd_rotate) g_rotate = nullptr;
decltype(&kvd_rotate_append_paged) g_rotate_append = nullptr;
decltype(&kvd_attend_paged_prefix_workspace_bytes) g_prefix_workspace = nullptr;
decltype(&kvd_attend_paged_prefix) g_prefix = nullptr;
decltype(&kvd_sample) g_sample = nullptr;
decltype(&kvd_filter_probs) g_filter = nullptr;
PyObject* g_check = nullptr;  // kvd._check(name, status): raises

// A Python exception that is set already.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& text) {
    PyErr_SetString(type, text.c_str());
    throw Raised{};
}

using Shape = std::initializer_list<int64_t>;

std::string text(at::IntArrayRef s) {
    std::string t = "[";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + "]";
}

const char* type_name(at::ScalarType t) { return c10::toString(t); }

// One call's view of its arguments.
struct Call {
    const char* fn;
    int dev = -1;
    PyObject* const* args;

    std::string where(const char* name) const { return std::string(fn) + ": " + name; }

    const at::Tensor& tensor(int i, const char* name) const {
        if (!THPVariable_Check(args[i])) raise(PyExc_TypeError, where(name) + " must be a tensor");
        return THPVariable_Unpack(args[i]);
    }
    bool given(int i) const { return args[i] != Py_None; }

    // The first tensor decides the device.
    const at::Tensor& first(int i, const char* name, int dims, const char* form) {
        const at::Tensor& t = tensor(i, name);
        if (t.dim() != dims) raise(PyExc_ValueError, where(name) + " must be " + form);
        if (!t.is_cuda()) raise(PyExc_ValueError, where(name) + " must be a contiguous CUDA tensor");
        dev = t.get_device();
        return t;
    }

    // The data pointer of a contiguous tensor of the call's device, this type and
    // shape.
    void* data(const at::Tensor& t, const char* name, at::ScalarType dtype, Shape shape) const {
        if (!t.is_cuda() || !t.is_contiguous())
            raise(PyExc_ValueError, where(name) + " must be a contiguous CUDA tensor");
        if (t.get_device() != dev)
            raise(PyExc_ValueError, where(name) + " is on cuda:" + std::to_string(t.get_device()) +
                                        ", not on cuda:" + std::to_string(dev));
        if (t.scalar_type() != dtype)
            raise(PyExc_TypeError, where(name) + " must be " + type_name(dtype) + ", not " +
                                       type_name(t.scalar_type()));
        if (t.sizes() != at::IntArrayRef(shape.begin(), shape.size()))
            raise(PyExc_ValueError, where(name) + " must be " +
                                        text(at::IntArrayRef(shape.begin(), shape.size())) +
                                        ", not " + text(t.sizes()));
        return t.data_ptr();
    }
    void* data(int i, const char* name, at::ScalarType dtype, Shape shape) const {
        return data(tensor(i, name), name, dtype, shape);
    }
    void* maybe(int i, const char* name, at::ScalarType dtype, Shape shape) const {
        return given(i) ? data(i, name, dtype, shape) : nullptr;
    }
    // An output that was passed, or a new one.
    at::Tensor output(int i, const char* name, at::ScalarType dtype, Shape shape) const {
        if (given(i)) {
            const at::Tensor& t = tensor(i, name);
            data(t, name, dtype, shape);
            return t;
        }
        return at::empty(at::IntArrayRef(shape.begin(), shape.size()),
                         at::TensorOptions().dtype(dtype).device(at::kCUDA, (c10::DeviceIndex)dev));
    }
    // New int32 outputs in one allocation, each from a 256-byte boundary of it (an allocation
    // takes the host a microsecond, such a view a tenth of one).
    template <size_t K>
    std::array<at::Tensor, K> outputs(const int64_t (&lengths)[K]) const {
        int64_t total = 0;
        for (int64_t n : lengths) total += (n + 63) / 64 * 64;
        const at::Tensor all = at::empty(
            {total}, at::TensorOptions().dtype(at::kInt).device(at::kCUDA, (c10::DeviceIndex)dev));
        std::array<at::Tensor, K> out;
        int64_t at = 0;
        for (size_t i = 0; i < K; ++i) {
            out[i] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()),
                                                              all.key_set(), all.dtype());
            out[i].unsafeGetTensorImpl()->set_storage_offset(at);
            out[i].unsafeGetTensorImpl()->set_sizes_contiguous(lengths[i]);
            at += (lengths[i] + 63) / 64 * 64;
        }
        return out;
    }
    int32_t* status(int i) const {
        if (!given(i)) return nullptr;
        const at::Tensor& t = tensor(i, "dev_status");
        if (t.numel() < 1) raise(PyExc_ValueError, where("dev_status") + " must hold a word");
        if (!t.is_cuda() || !t.is_contiguous() || t.get_device() != dev ||
            t.scalar_type() != at::kInt)
            raise(PyExc_ValueError, where("dev_status") + " must be an int32 CUDA tensor of cuda:" +
                                        std::to_string(dev));
        return static_cast<int32_t*>(t.data_ptr());
    }
    kvd_dtype code(at::ScalarType t) const {
        if (t == at::kBFloat16) return KVD_BF16;
        if (t == at::kFloat) return KVD_F32;
        raise(PyExc_TypeError,
              std::string(fn) + ": unsupported dtype " + type_name(t) + " (bf16 or fp32)");
    }
    float number(int i) const {
        const double x = PyFloat_AsDouble(args[i]);
        if (x == -1.0 && PyErr_Occurred()) throw Raised{};
        return (float)x;
    }
    int whole(int i, const char* name) const {
        const long long x = PyLong_AsLongLong(args[i]);
        if (x == -1 && PyErr_Occurred()) throw Raised{};
        if (x < INT32_MIN) raise(PyExc_ValueError, where(name) + " does not fit 32 bits");
        return small(x, name);
    }
    bool truth(int i) const {
        const int x = PyObject_IsTrue(args[i]);
        if (x < 0) throw Raised{};
        return x != 0;
    }
    // A tensor's first extent, for arguments whose length sets others'.
    int64_t length(int i, const char* name, int dims, const char* form) const {
        const at::Tensor& t = tensor(i, name);
        if (t.dim() != dims) raise(PyExc_ValueError, where(name) + " must be " + form);
        return t.size(0);
    }
    at::Tensor scratch(int i, size_t bytes) const {
        if (given(i)) {
            const at::Tensor& t = tensor(i, "workspace");
            if (!t.is_cuda() || !t.is_contiguous() || t.get_device() != dev)
                raise(PyExc_ValueError, where("workspace") +
                                            " must be a contiguous CUDA tensor of the call's device");
            return t;
        }
        return at::empty({(int64_t)bytes}, at::TensorOptions().dtype(at::kByte).device(
                                               at::kCUDA, (c10::DeviceIndex)dev));
    }
    int small(int64_t x, const char* name) const {
        if (x > INT32_MAX) raise(PyExc_ValueError, where(name) + " does not fit 32 bits");
        return (int)x;
    }

    // The entry point, on the call's device and its current stream, without the
    // interpreter lock.
    template <typename F>
    void run(const char* entry, F f) const {
        kvd_status st;
        {
            c10::cuda::OptionalCUDAGuard guard;
            if (c10::cuda::current_device() != dev) guard.set_index((c10::DeviceIndex)dev);
            const auto stream =
                (kvd_stream_t)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
            Py_BEGIN_ALLOW_THREADS
            st = f(stream);
            Py_END_ALLOW_THREADS
        }
        if (st != KVD_OK) {
            PyObject* r = PyObject_CallFunction(g_check, "si", entry, (int)st);
            Py_XDECREF(r);
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, entry);
            throw Raised{};
        }
    }
};

constexpr auto kI32 = at::kInt;
constexpr auto kF32 = at::kFloat;

struct Cache {
    int64_t NB, BS, R, P;
    at::ScalarType dtype;
    void *latent, *rope;
};

Cache cache(Call& c, int i, int j) {
    const char* form = "[NB, BS, 1, R], the rotary one [NB, BS, 1, P]";
    const at::Tensor& l = c.first(i, "latent_cache", 4, form);
    const at::Tensor& r = c.tensor(j, "rope_cache");
    if (r.dim() != 4) raise(PyExc_ValueError, c.where("rope_cache") + " must be [NB, BS, 1, P]");
    Cache k{l.size(0), l.size(1), l.size(3), r.size(3), l.scalar_type(), nullptr, nullptr};
    k.latent = c.data(l, "latent_cache", k.dtype, {k.NB, k.BS, 1, k.R});
    k.rope = c.data(r, "rope_cache", k.dtype, {k.NB, k.BS, 1, k.P});
    return k;
}

int64_t columns(const Call& c, int i) {
    const at::Tensor& t = c.tensor(i, "block_tables");
    if (t.dim() != 2) raise(PyExc_ValueError, c.where("block_tables") + " must be int32 [Q, cols]");
    return t.size(1);
}

PyObject* append_latent(Call& c) {
    const Cache k = cache(c, 0, 1);
    const int64_t cols = columns(c, 2), Q = c.tensor(7, "pos").numel(),
                  N = c.tensor(4, "latent_new").dim() == 2 ? c.tensor(4, "latent_new").size(0) : -1;
    auto* tables = static_cast<const int32_t*>(c.data(2, "block_tables", kI32, {Q, cols}));
    auto* offset = static_cast<const int32_t*>(c.maybe(3, "seq_offset", kI32, {Q}));
    const void* ln = c.data(4, "latent_new", k.dtype, {N, k.R});
    const void* rn = c.data(5, "rope_new", k.dtype, {N, k.P});
    auto* lens = static_cast<const int32_t*>(c.data(6, "new_lens", kI32, {Q + 1}));
    auto* pos = static_cast<const int32_t*>(c.data(7, "pos", kI32, {Q}));
    int32_t* status = c.status(8);
    const kvd_dtype dt = c.code(k.dtype);
    const int q = c.small(Q, "pos"), n = c.small(N, "latent_new"), nb = c.small(k.NB, "latent_cache"),
              bs = c.small(k.BS, "latent_cache"), co = c.small(cols, "block_tables"),
              r = c.small(k.R, "latent_cache"), p = c.small(k.P, "rope_cache");
    c.run("kvd_append_latent", [&](kvd_stream_t s) {
        return g_append(k.latent, k.rope, ln, rn, tables, offset, lens, pos, q, n, nb, bs, co, r, p,
                        dt, status, s);
    });
    Py_RETURN_NONE;
}

PyObject* attend_latent(Call& c) {
    const Cache k = cache(c, 2, 3);
    const at::Tensor& ql = c.tensor(0, "q_latent");
    if (ql.dim() != 4)
        raise(PyExc_ValueError,
              std::string(c.fn) + ": queries must be [Q, T, H, R] and [Q, T, H, P]");
    const int64_t Q = ql.size(0), T = ql.size(1), H = ql.size(2), cols = columns(c, 4);
    const kvd_dtype dt = c.code(k.dtype);
    const void* lp = c.data(ql, "q_latent", k.dtype, {Q, T, H, k.R});
    const void* rp = c.data(1, "q_rope", k.dtype, {Q, T, H, k.P});
    auto* tables = static_cast<const int32_t*>(c.data(4, "block_tables", kI32, {Q, cols}));
    auto* lens = static_cast<const int32_t*>(c.data(5, "seq_lens", kI32, {Q + 1}));
    const float scale = c.number(6);
    auto* offset = static_cast<const int32_t*>(c.maybe(7, "seq_offset", kI32, {Q}));
    float* lse = static_cast<float*>(c.maybe(9, "lse", kF32, {Q, T, H}));
    int32_t* status = c.status(11);
    const int q = c.small(Q, "q_latent"), t = c.small(T, "q_latent"), h = c.small(H, "q_latent"),
              nb = c.small(k.NB, "latent_cache"), bs = c.small(k.BS, "latent_cache"),
              co = c.small(cols, "block_tables"), r = c.small(k.R, "latent_cache"),
              p = c.small(k.P, "rope_cache");
    at::Tensor out = c.output(8, "out", k.dtype, {Q, T, H, k.R}), ws;
    if (c.given(10)) {
        ws = c.tensor(10, "workspace");
        if (!ws.is_cuda() || !ws.is_contiguous() || ws.get_device() != c.dev)
            raise(PyExc_ValueError, c.where("workspace") +
                                        " must be a contiguous CUDA tensor of the call's device");
    } else {
        ws = at::empty({(int64_t)g_workspace(q, t, h, bs, co, r, p, dt)},
                       at::TensorOptions().dtype(at::kByte).device(at::kCUDA,
                                                                   (c10::DeviceIndex)c.dev));
    }
    c.run("kvd_attend_latent", [&](kvd_stream_t s) {
        return g_attend(lp, rp, k.latent, k.rope, tables, lens, offset, out.data_ptr(), lse, q, t, h,
                        nb, bs, co, r, p, scale, dt, ws.data_ptr(), ws.nbytes(), status, s);
    });
    return THPVariable_Wrap(out);
}

PyObject* attend_expanded(Call& c) {
    const at::Tensor& q = c.first(0, "q", 3, "[Nq, H, Dn + P]");
    const at::Tensor &kv = c.tensor(1, "kv"), &kr = c.tensor(2, "k_rope");
    if (kv.dim() != 3 || kr.dim() != 2)
        raise(PyExc_ValueError, std::string(c.fn) + ": kv [Nk, H, Dn + Dv], k_rope [Nk, P] required");
    const at::ScalarType dtype = q.scalar_type();
    const int64_t Nq = q.size(0), H = q.size(1), Nk = kr.size(0), P = kr.size(1),
                  Dn = q.size(2) - P, Dv = kv.size(2) - Dn, Q = c.tensor(3, "q_lens").numel() - 1;
    if (Dn < 1 || Dv < 1)
        raise(PyExc_ValueError, std::string(c.fn) + ": rows of q " + std::to_string(q.size(2)) +
                                    ", kv " + std::to_string(kv.size(2)) + " and k_rope " +
                                    std::to_string(P) + " do not fit");
    const kvd_dtype dt = c.code(dtype);
    const void* qp = c.data(q, "q", dtype, {Nq, H, Dn + P});
    const void* kp = c.data(kv, "kv", dtype, {Nk, H, Dn + Dv});
    const void* rp = c.data(kr, "k_rope", dtype, {Nk, P});
    auto* ql = static_cast<const int32_t*>(c.data(3, "q_lens", kI32, {Q + 1}));
    auto* kl = static_cast<const int32_t*>(c.data(4, "k_lens", kI32, {Q + 1}));
    const float scale = c.number(5);
    const int causal = PyObject_IsTrue(c.args[6]);
    if (causal < 0) throw Raised{};
    float* lse = static_cast<float*>(c.maybe(8, "lse", kF32, {Nq, H}));
    int32_t* status = c.status(9);
    const int nq = c.small(Nq, "q"), nk = c.small(Nk, "kv"), h = c.small(H, "q"),
              n = c.small(Q, "q_lens"), dn = c.small(Dn, "q"), dv = c.small(Dv, "kv"),
              p = c.small(P, "k_rope");
    at::Tensor out = c.output(7, "out", dtype, {Nq, H, Dv});
    c.run("kvd_attend_expanded", [&](kvd_stream_t s) {
        return g_expanded(qp, kp, rp, ql, kl, out.data_ptr(), lse, n, nq, nk, h, dn, dv, p, scale,
                          causal, dt, status, s);
    });
    return THPVariable_Wrap(out);
}

PyObject* verify_drafts(Call& c) {
    const at::Tensor& tp = c.first(0, "target_probs", 3, "[Q, T + 1, V]");
    const at::ScalarType dtype = tp.scalar_type();
    const int64_t Q = tp.size(0), T = tp.size(1) - 1, V = tp.size(2);
    if (T < 0) raise(PyExc_ValueError, c.where("target_probs") + " must be [Q, T + 1, V]");
    const kvd_dtype dt = c.code(dtype);
    const void* pp = c.data(tp, "target_probs", dtype, {Q, T + 1, V});
    const void* dp = nullptr;
    const int32_t* xp = nullptr;
    const float* up = nullptr;
    if (T > 0) {
        dp = c.data(1, "draft_probs", dtype, {Q, T, V});
        xp = static_cast<const int32_t*>(c.data(2, "draft_tokens", kI32, {Q, T}));
        up = static_cast<const float*>(c.data(3, "u_accept", kF32, {Q, T}));
    }
    auto* sp = static_cast<const float*>(c.data(4, "u_sample", kF32, {Q}));
    auto* mp = static_cast<const int32_t*>(c.maybe(5, "num_drafts", kI32, {Q}));
    int32_t* status = c.status(8);
    const int q = c.small(Q, "target_probs"), t = c.small(T, "target_probs"),
              v = c.small(V, "target_probs");
    at::Tensor tokens = c.output(6, "tokens", kI32, {Q, T + 1});
    at::Tensor accepted = c.output(7, "accepted", kI32, {Q});
    c.run("kvd_verify_drafts", [&](kvd_stream_t s) {
        return g_verify(pp, dp, xp, up, sp, mp, static_cast<int32_t*>(tokens.data_ptr()),
                        static_cast<int32_t*>(accepted.data_ptr()), q, t, v, dt, status, s);
    });
    PyObject* a = THPVariable_Wrap(tokens);
    PyObject* b = a ? THPVariable_Wrap(accepted) : nullptr;
    if (!b) {
        Py_XDECREF(a);
        throw Raised{};
    }
    PyObject* r = PyTuple_Pack(2, a, b);
    Py_DECREF(a);
    Py_DECREF(b);
    return r;
}

PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) throw Raised{};
    Py_ssize_t i = 0;
    for (const at::Tensor& t : ts) {
        PyObject* o = THPVariable_Wrap(t);
        if (!o) {
            Py_DECREF(r);
            throw Raised{};
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

int32_t* ints(void* p) { return static_cast<int32_t*>(p); }
float* floats(void* p) { return static_cast<float*>(p); }

PyObject* plan_pages(Call& c) {
    const at::Tensor& bt = c.first(0, "block_tables", 2, "int32 [Q, cols]");
    const int64_t Q = bt.size(0), cols = bt.size(1), F = c.length(2, "free_pages", 1, "int32 [F]");
    int32_t* tables = ints(c.data(bt, "block_tables", kI32, {Q, cols}));
    int32_t* held = ints(c.data(1, "pages_held", kI32, {Q}));
    int32_t* pages = ints(c.data(2, "free_pages", kI32, {F}));
    int32_t* count = ints(c.data(3, "free_count", kI32, {1}));
    const int32_t* kept = ints(c.data(4, "kept_lens", kI32, {Q}));
    const int32_t* lens = ints(c.data(5, "new_lens", kI32, {Q + 1}));
    const int bs = c.whole(6, "block_size"), n = c.whole(7, "num_tokens");
    if (n < 0) raise(PyExc_ValueError, c.where("num_tokens") + " must not be negative");
    const int32_t* base = ints(c.maybe(8, "pos_base", kI32, {Q}));
    int32_t* status = c.status(12);
    const int q = c.small(Q, "block_tables"), co = c.small(cols, "block_tables"),
              f = c.small(F, "free_pages");
    at::Tensor sl, st, ps;
    if (!c.given(9) && !c.given(10) && !c.given(11)) {
        auto o = c.outputs<3>({Q + 1, n, n});
        sl = o[0], st = o[1], ps = o[2];
    } else {
        sl = c.output(9, "seq_lens", kI32, {Q + 1});
        st = c.output(10, "slots", kI32, {n});
        ps = c.output(11, "positions", kI32, {n});
    }
    c.run("kvd_plan_pages", [&](kvd_stream_t s) {
        return g_plan_pages(tables, held, pages, count, kept, lens, base, ints(sl.data_ptr()),
                            ints(st.data_ptr()), ints(ps.data_ptr()), q, n, bs, co, f, status, s);
    });
    return tuple_of({sl, st, ps});
}

PyObject* rotate(Call& c) {
    const at::Tensor& x = c.first(0, "x", 3, "[N, H, D]");
    const at::ScalarType dtype = x.scalar_type();
    const int64_t N = x.size(0), H = x.size(1), D = x.size(2),
                  F = c.length(2, "freqs", 1, "float64 [Dr / 2]");
    const kvd_dtype dt = c.code(dtype);
    const void* xp = c.data(x, "x", dtype, {N, H, D});
    const int32_t* pos = ints(c.data(1, "positions", kI32, {N}));
    auto* freqs = static_cast<const double*>(c.data(2, "freqs", at::kDouble, {F}));
    const void* w = c.maybe(3, "weight", dtype, {D});
    const float eps = c.number(4), scale = c.number(6);
    const bool inter = c.truth(5);
    int32_t* status = c.status(8);
    const int n = c.small(N, "x"), h = c.small(H, "x"), d = c.small(D, "x"),
              dr = c.small(2 * F, "freqs");
    at::Tensor out = c.output(7, "out", dtype, {N, H, D});
    c.run("kvd_rotate", [&](kvd_stream_t s) {
        return g_rotate(xp, w, freqs, pos, out.data_ptr(), n, h, d, dr, inter, scale, eps, dt,
                        status, s);
    });
    return THPVariable_Wrap(out);
}

PyObject* rotate_append_paged(Call& c) {
    const at::Tensor& x = c.first(0, "qkv", 3, "[N, Hq + 2 Hkv, D]");
    const at::Tensor &kc = c.tensor(1, "key_cache"), &vc = c.tensor(2, "value_cache");
    if (kc.dim() != 4) raise(PyExc_ValueError, c.where("key_cache") + " must be [NB, BS, Hkv, D]");
    const at::ScalarType dtype = x.scalar_type();
    const int64_t N = x.size(0), NB = kc.size(0), BS = kc.size(1), Hkv = kc.size(2), D = kc.size(3),
                  Hq = x.size(1) - 2 * Hkv, F = c.length(5, "freqs", 1, "float64 [Dr / 2]");
    if (Hq < 1)
        raise(PyExc_ValueError, c.where("qkv") + " has " + std::to_string(x.size(1)) +
                                    " heads, " + std::to_string(Hkv) + " of them keys and " +
                                    std::to_string(Hkv) + " values");
    const kvd_dtype dt = c.code(dtype);
    const void* xp = c.data(x, "qkv", dtype, {N, Hq + 2 * Hkv, D});
    void* kp = c.data(kc, "key_cache", dtype, {NB, BS, Hkv, D});
    void* vp = c.data(vc, "value_cache", dtype, {NB, BS, Hkv, D});
    const int32_t* slots = ints(c.data(3, "slots", kI32, {N}));
    const int32_t* pos = ints(c.data(4, "positions", kI32, {N}));
    auto* freqs = static_cast<const double*>(c.data(5, "freqs", at::kDouble, {F}));
    const void* qw = c.maybe(6, "q_weight", dtype, {D});
    const void* kw = c.maybe(7, "k_weight", dtype, {D});
    const float eps = c.number(8), scale = c.number(10);
    const bool inter = c.truth(9);
    int32_t* status = c.status(12);
    const int n = c.small(N, "qkv"), hq = c.small(Hq, "qkv"), hk = c.small(Hkv, "key_cache"),
              nb = c.small(NB, "key_cache"), bs = c.small(BS, "key_cache"),
              d = c.small(D, "key_cache"), dr = c.small(2 * F, "freqs");
    at::Tensor out = c.output(11, "out", dtype, {N, Hq, D});
    c.run("kvd_rotate_append_paged", [&](kvd_stream_t s) {
        return g_rotate_append(xp, qw, kw, freqs, pos, slots, out.data_ptr(), kp, vp, n, hq, hk, nb,
                               bs, d, dr, inter, scale, eps, dt, status, s);
    });
    return THPVariable_Wrap(out);
}

PyObject* attend_paged_prefix(Call& c) {
    const at::Tensor& q = c.first(0, "q", 3, "[Q, Hq, D]");
    const at::Tensor &kc = c.tensor(1, "key_cache"), &vc = c.tensor(2, "value_cache"),
                     &pt = c.tensor(3, "prefix_tables");
    if (kc.dim() != 4) raise(PyExc_ValueError, c.where("key_cache") + " must be [NB, BS, Hkv, D]");
    if (pt.dim() != 2) raise(PyExc_ValueError, c.where("prefix_tables") + " must be int32 [G, pcols]");
    const at::ScalarType dtype = q.scalar_type();
    const int64_t Q = q.size(0), Hq = q.size(1), D = q.size(2), NB = kc.size(0), BS = kc.size(1),
                  Hkv = kc.size(2), G = pt.size(0), pcols = pt.size(1), cols = columns(c, 6);
    const kvd_dtype dt = c.code(dtype);
    const void* qp = c.data(q, "q", dtype, {Q, Hq, D});
    const void* kp = c.data(kc, "key_cache", dtype, {NB, BS, Hkv, D});
    const void* vp = c.data(vc, "value_cache", dtype, {NB, BS, Hkv, D});
    const int32_t* pp = ints(c.data(pt, "prefix_tables", kI32, {G, pcols}));
    const int32_t* pl = ints(c.data(4, "prefix_lens", kI32, {G}));
    const int32_t* gl = ints(c.data(5, "group_lens", kI32, {G + 1}));
    const int32_t* tables = ints(c.data(6, "block_tables", kI32, {Q, cols}));
    const int32_t* lens = ints(c.data(7, "seq_lens", kI32, {Q + 1}));
    const int32_t* offset = ints(c.maybe(8, "seq_offset", kI32, {Q}));
    const float scale = c.number(9);
    float* lse = floats(c.maybe(11, "lse", kF32, {Q, Hq}));
    int32_t* status = c.status(13);
    const int n = c.small(Q, "q"), g = c.small(G, "prefix_tables"), hq = c.small(Hq, "q"),
              hk = c.small(Hkv, "key_cache"), nb = c.small(NB, "key_cache"),
              bs = c.small(BS, "key_cache"), pc = c.small(pcols, "prefix_tables"),
              co = c.small(cols, "block_tables"), d = c.small(D, "q");
    at::Tensor out = c.output(10, "out", dtype, {Q, Hq, D});
    at::Tensor ws = c.scratch(12, c.given(12) ? 0 : g_prefix_workspace(n, g, hq, hk, bs, pc, co, d, dt));
    c.run("kvd_attend_paged_prefix", [&](kvd_stream_t s) {
        return g_prefix(qp, kp, vp, pp, pl, gl, tables, lens, offset, out.data_ptr(), lse, n, g, hq,
                        hk, nb, bs, pc, co, d, scale, dt, ws.data_ptr(), ws.nbytes(), status, s);
    });
    return THPVariable_Wrap(out);
}

PyObject* sample_rows(Call& c) {
    const at::Tensor& l = c.first(0, "logits", 2, "[R, V]");
    const at::ScalarType dtype = l.scalar_type();
    const int64_t R = l.size(0), V = l.size(1);
    const kvd_dtype dt = c.code(dtype);
    const void* lp = c.data(l, "logits", dtype, {R, V});
    const float* u = floats(c.data(1, "u", kF32, {R}));
    const float* temp = floats(c.maybe(2, "temperature", kF32, {R}));
    const int32_t* k = ints(c.maybe(3, "top_k", kI32, {R}));
    const float* p = floats(c.maybe(4, "top_p", kF32, {R}));
    const float* m = floats(c.maybe(5, "min_p", kF32, {R}));
    int32_t* status = c.status(7);
    const int r = c.small(R, "logits"), v = c.small(V, "logits");
    at::Tensor tokens = c.output(6, "tokens", kI32, {R});
    c.run("kvd_sample", [&](kvd_stream_t s) {
        return g_sample(lp, temp, k, p, m, u, ints(tokens.data_ptr()), r, v, dt, status, s);
    });
    return THPVariable_Wrap(tokens);
}

PyObject* filter_probs(Call& c) {
    const at::Tensor& l = c.first(0, "logits", 2, "[R, V]");
    const at::ScalarType dtype = l.scalar_type();
    const int64_t R = l.size(0), V = l.size(1);
    const kvd_dtype dt = c.code(dtype);
    const void* lp = c.data(l, "logits", dtype, {R, V});
    const float* temp = floats(c.maybe(1, "temperature", kF32, {R}));
    const int32_t* k = ints(c.maybe(2, "top_k", kI32, {R}));
    const float* p = floats(c.maybe(3, "top_p", kF32, {R}));
    const float* m = floats(c.maybe(4, "min_p", kF32, {R}));
    const at::ScalarType to = c.given(5) ? c.tensor(5, "out").scalar_type() : dtype;
    const kvd_dtype pt = c.code(to);
    int32_t* status = c.status(6);
    const int r = c.small(R, "logits"), v = c.small(V, "logits");
    at::Tensor out = c.output(5, "out", to, {R, V});
    c.run("kvd_filter_probs", [&](kvd_stream_t s) {
        return g_filter(lp, temp, k, p, m, out.data_ptr(), r, v, dt, pt, status, s);
    });
    return THPVariable_Wrap(out);
}

// No C++ exception leaves a call.
template <PyObject* (*F)(Call&), int N>
PyObject* guarded(const char* fn, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%s: %d arguments expected, %zd given", fn, N, n);
        return nullptr;
    }
    if (!g_check) {
        PyErr_SetString(PyExc_RuntimeError, "bind() first");
        return nullptr;
    }
    Call c{fn, -1, args};
    try {
        return F(c);
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded<append_latent, 9>("append_latent", a, n);
}
PyObject* py_attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded<attend_latent, 12>("attend_latent", a, n);
}
PyObject* py_expanded(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded<attend_expanded, 10>("attend_expanded", a, n);
}
PyObject* py_verify(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded<verify_drafts, 9>("verify_drafts", a, n);
}

PyObject* py_plan_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded<plan_pages, 13>("plan_pages", a, n);
}
PyObject* py_rotate(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded<rotate, 9>("rotate", a, n);
}
PyObject* py_rotate_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded<rotate_append_paged, 13>("rotate_append_paged", a, n);
}
PyObject* py_prefix(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded<attend_paged_prefix, 14>("attend_paged_prefix", a, n);
}
PyObject* py_sample(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded<sample_rows, 8>("sample", a, n);
}
PyObject* py_filter(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded<filter_probs, 7>("filter_probs", a, n);
}

// bind(check, twelve addresses): the entry points of the loaded library.
PyObject* py_bind(PyObject*, PyObject* args) {
    PyObject* check;
    unsigned long long f[12];
    if (!PyArg_ParseTuple(args, "OKKKKKKKKKKKK", &check, f, f + 1, f + 2, f + 3, f + 4, f + 5, f + 6,
                          f + 7, f + 8, f + 9, f + 10, f + 11))
        return nullptr;
    g_append = reinterpret_cast<decltype(g_append)>(f[0]);
    g_workspace = reinterpret_cast<decltype(g_workspace)>(f[1]);
    g_attend = reinterpret_cast<decltype(g_attend)>(f[2]);
    g_expanded = reinterpret_cast<decltype(g_expanded)>(f[3]);
    g_verify = reinterpret_cast<decltype(g_verify)>(f[4]);
    g_plan_pages = reinterpret_cast<decltype(g_plan_pages)>(f[5]);
    g_rotate = reinterpret_cast<decltype(g_rotate)>(f[6]);
    g_rotate_append = reinterpret_cast<decltype(g_rotate_append)>(f[7]);
    g_prefix_workspace = reinterpret_cast<decltype(g_prefix_workspace)>(f[8]);
    g_prefix = reinterpret_cast<decltype(g_prefix)>(f[9]);
    g_sample = reinterpret_cast<decltype(g_sample)>(f[10]);
    g_filter = reinterpret_cast<decltype(g_filter)>(f[11]);
    Py_INCREF(check);
    Py_XSETREF(g_check, check);
    Py_RETURN_NONE;
}

#define FAST(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {
    {"bind", py_bind, METH_VARARGS, nullptr},
    FAST("append_latent", py_append),
    FAST("attend_latent", py_attend),
    FAST("attend_expanded", py_expanded),
    FAST("verify_drafts", py_verify),
    FAST("plan_pages", py_plan_pages),
    FAST("rotate", py_rotate),
    FAST("rotate_append_paged", py_rotate_append),
    FAST("attend_paged_prefix", py_prefix),
    FAST("sample", py_sample),
    FAST("filter_probs", py_filter),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_latent_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__latent_binding() { return PyModule_Create(&g_module); }
