// latent_binding.cpp -- the latent-cache calls of kvd.py, from torch tensors to
// the C entry points: argument checks, outputs, device and stream.  A decode loop
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

#include <initializer_list>
#include <string>

#include "../../../include/kvd.h"

namespace {

decltype(&kvd_append_latent) g_append = nullptr;
decltype(&kvd_attend_latent_workspace_bytes) g_workspace = nullptr;
decltype(&kvd_attend_latent) g_attend = nullptr;
decltype(&kvd_attend_expanded) g_expanded = nullptr;
decltype(&kvd_verify_drafts) g_verify = nullptr;
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

// bind(check, five addresses): the entry points of the loaded library.
PyObject* py_bind(PyObject*, PyObject* args) {
    PyObject* check;
    unsigned long long f[5];
    if (!PyArg_ParseTuple(args, "OKKKKK", &check, f, f + 1, f + 2, f + 3, f + 4)) return nullptr;
    g_append = reinterpret_cast<decltype(g_append)>(f[0]);
    g_workspace = reinterpret_cast<decltype(g_workspace)>(f[1]);
    g_attend = reinterpret_cast<decltype(g_attend)>(f[2]);
    g_expanded = reinterpret_cast<decltype(g_expanded)>(f[3]);
    g_verify = reinterpret_cast<decltype(g_verify)>(f[4]);
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
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_latent_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__latent_binding() { return PyModule_Create(&g_module); }
