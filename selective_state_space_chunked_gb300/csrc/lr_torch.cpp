// lr_torch.cpp -- the short path of the torch helpers that are called once per
// layer and token, where the GPU's own time is a few microseconds: argument
// checks, result allocation and the call of the C ABI without the interpreter
// between them (host time of a step 16 -> 3.6 us, of a prompt 21 -> 6.9, of a group norm
// 12 -> 3.6).
//
// Each function takes what its helper in binding.py takes and returns what it
// returns, or None where an argument is not already what the kernels take
// (another type or device, not contiguous or in rows that are not evenly apart, shapes
// that do not match, empty; the selective scan with heads copies what only stands in the
// wrong place) or the call's own checks refused it; nothing has been launched then, and the helper
// goes on to its own checks and conversions, which convert the argument or say what
// is wrong.  Any other status comes back as an int, for the helper to raise: part of
// the call may have run, and it may have updated a state in place.  The interpreter
// is released for the allocations and the call: both may wait for the GPU.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <vector>

#include "lrscan.h"

namespace {

// A GPU and a dtype that the tensors of a call have to share.
struct Call {
    c10::DeviceIndex dev = -1;
    at::ScalarType type = at::kFloat;
    lr_dtype io = LR_F32;

    // the first tensor names both
    const at::Tensor *first(PyObject *o) {
        if (!THPVariable_CheckExact(o)) return nullptr;
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.layout() != at::kStrided || !t.is_contiguous() || t.numel() == 0) return nullptr;
        type = t.scalar_type();
        if (type != at::kFloat && type != at::kBFloat16) return nullptr;
        io = type == at::kBFloat16 ? LR_BF16 : LR_F32;
        dev = t.get_device();
        return dev == c10::cuda::current_device() ? &t : nullptr;
    }
    // a tensor of the given shape; None gives a null pointer where that is allowed
    bool take(PyObject *o, at::ScalarType want, at::IntArrayRef shape, bool optional, void **p) const {
        if (o == Py_None) {
            *p = nullptr;
            return optional;
        }
        if (!THPVariable_CheckExact(o)) return false;
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.layout() != at::kStrided || t.get_device() != dev || t.scalar_type() != want ||
            t.sizes() != shape || !t.is_contiguous())
            return false;
        *p = t.data_ptr();
        return true;
    }
    // a tensor of the given shape, of the call's GPU and dtype
    bool like(PyObject *o, at::IntArrayRef shape) const {
        if (!THPVariable_CheckExact(o)) return false;
        const at::Tensor &t = THPVariable_Unpack(o);
        return t.is_cuda() && t.layout() == at::kStrided && t.get_device() == dev && t.scalar_type() == type &&
               t.sizes() == shape;
    }
    // a tensor whose rows of `width` lie evenly apart (a slice of a wider one): the elements
    // from one to the next.  whole: on 16-byte boundaries, unless they are dense.
    bool rows(PyObject *o, bool whole, bool optional, void **p, int64_t *ld, at::IntArrayRef shape) const {
        if (o == Py_None) {
            *p = nullptr, *ld = 0;
            return optional;
        }
        if (!like(o, shape)) return false;
        const at::Tensor &t = THPVariable_Unpack(o);
        *ld = pitch(t);
        *p = t.data_ptr();
        return *ld > 0 && reinterpret_cast<uintptr_t>(*p) % 16 == 0 &&
               (!whole || *ld == t.size(-1) || *ld * t.element_size() % 16 == 0);
    }
    // ... which names the call's GPU and dtype
    const at::Tensor *first_rows(PyObject *o, int64_t dims) {
        if (!THPVariable_CheckExact(o)) return nullptr;
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.layout() != at::kStrided || t.numel() == 0 || (dims > 0 && t.dim() != dims) || t.dim() < 1)
            return nullptr;
        type = t.scalar_type();
        if (type != at::kFloat && type != at::kBFloat16) return nullptr;
        io = type == at::kBFloat16 ? LR_BF16 : LR_F32;
        dev = t.get_device();
        return dev == c10::cuda::current_device() ? &t : nullptr;
    }
    // elements between the rows of t (..., C), 0 where they are not evenly apart
    static int64_t pitch(const at::Tensor &t) {
        const int64_t n = t.dim(), C = t.size(-1);
        if (C != 1 && t.stride(-1) != 1) return 0;
        int64_t ld = -1, size = 1;
        for (int64_t i = n - 2; i >= 0; --i) {
            if (t.size(i) == 1) continue;
            if (ld < 0)
                ld = t.stride(i);
            else if (t.stride(i) != ld * size)
                return 0;
            size *= t.size(i);
        }
        return ld < 0 ? C : ld < C ? 0 : ld;
    }
    lr_stream_t stream() const {
        return reinterpret_cast<lr_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream());
    }
};

bool to_int(PyObject *o, int64_t *v) {
    *v = PyLong_AsLongLong(o);
    if (*v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    return true;
}
bool to_float(PyObject *o, float *v) {
    const double d = PyFloat_AsDouble(o);
    if (d == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    *v = static_cast<float>(d);
    return true;
}

// Sizes of q, k (..., Hk dk) and v (..., H dv).
struct Heads {
    int64_t H, Hk, dk, dv;
    bool of(PyObject *h, PyObject *hk, const at::Tensor &q, const at::Tensor &v) {
        if (!to_int(h, &H) || H < 1) return false;
        Hk = H;
        if (hk != Py_None && (!to_int(hk, &Hk) || Hk < 1 || H % Hk != 0)) return false;
        if (v.dim() != q.dim() || q.size(-1) % Hk != 0 || v.size(-1) % H != 0) return false;
        dk = q.size(-1) / Hk, dv = v.size(-1) / H;
        return dk > 0 && dv > 0;
    }
};

// An owned reference.
struct Ref {
    PyObject *o;
    explicit Ref(PyObject *p) : o(p) {}
    Ref(const Ref &) = delete;
    ~Ref() { Py_XDECREF(o); }
    static PyObject *share(PyObject *p) {
        Py_INCREF(p);
        return p;
    }
};

// The interpreter released while it lives.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    Unlocked() = default;
    Unlocked(const Unlocked &) = delete;
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// After a C++ exception: before the launch it is the helper's turn (an allocation
// that failed: its own says so), after it there is nothing to try again.
PyObject *thrown(bool launched) {
    if (!launched) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "the call ran, its results could not be returned");
    return nullptr;
}

// What a call that was not LR_OK gives: None after the checks that come before
// every launch, else the status.
PyObject *refused(int rc) {
    if (rc == LR_ERR_INVALID_ARG || rc == LR_ERR_UNSUPPORTED || rc == LR_ERR_MISALIGNED) Py_RETURN_NONE;
    return PyLong_FromLong(rc);
}

// (q, k, v, H, Hk, a_log, g, S, S_out, scale) -> (o, S_new)
PyObject *decay_attn_step(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 10) Py_RETURN_NONE;
    bool launched = false;
    try {
        Call c;
        Heads s;
        const at::Tensor *q = c.first(args[0]);
        if (q == nullptr || q->dim() != 2 || !THPVariable_CheckExact(args[2])) Py_RETURN_NONE;
        const at::Tensor &vt = THPVariable_Unpack(args[2]);
        if (!s.of(args[3], args[4], *q, vt)) Py_RETURN_NONE;
        const int64_t B = q->size(0);
        const int64_t vs[] = {B, s.H * s.dv}, gs[] = {B, s.H}, ss[] = {B, s.H, s.dv, s.dk};
        void *k, *v, *a, *g, *S_in, *S_out;
        float scale;
        if (!c.take(args[1], c.type, q->sizes(), false, &k) || !c.take(args[2], c.type, vs, false, &v) ||
            !c.take(args[5], at::kFloat, {s.H}, true, &a) || !c.take(args[6], c.type, gs, true, &g) ||
            !c.take(args[7], at::kFloat, ss, true, &S_in) || !c.take(args[8], at::kFloat, ss, true, &S_out) ||
            !to_float(args[9], &scale))
            Py_RETURN_NONE;
        at::Tensor o, Sn;
        int rc;
        {
            const Unlocked unlocked;
            o = at::empty(vs, q->options());
            if (S_out == nullptr) {
                Sn = at::empty(ss, q->options().dtype(at::kFloat));
                S_out = Sn.data_ptr();
            }
            launched = true;
            rc = lr_decay_attn_step(q->data_ptr(), k, v, static_cast<float *>(a), g, scale, static_cast<float *>(S_in),
                                    static_cast<float *>(S_out), o.data_ptr(), B, s.H, s.Hk, s.dk, s.dv, c.io,
                                    c.stream());
        }
        if (rc != LR_OK) return refused(rc);
        const Ref po(THPVariable_Wrap(o)), ps(Sn.defined() ? THPVariable_Wrap(Sn) : Ref::share(args[8]));
        return po.o && ps.o ? PyTuple_Pack(2, po.o, ps.o) : nullptr;
    } catch (...) {
        return thrown(launched);
    }
}

// (q, k, v, H, Hk, a_log, g, S0, lens, scale) -> (o, S_final, workspace)
PyObject *decay_attn(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 10) Py_RETURN_NONE;
    bool launched = false;
    try {
        Call c;
        Heads s;
        const at::Tensor *q = c.first(args[0]);
        if (q == nullptr || q->dim() != 3 || !THPVariable_CheckExact(args[2])) Py_RETURN_NONE;
        const at::Tensor &vt = THPVariable_Unpack(args[2]);
        if (!s.of(args[3], args[4], *q, vt)) Py_RETURN_NONE;
        const int64_t B = q->size(0), L = q->size(1);
        const int64_t vs[] = {B, L, s.H * s.dv}, gs[] = {B, L, s.H}, ss[] = {B, s.H, s.dv, s.dk};
        void *k, *v, *a, *g, *S0, *lens;
        float scale;
        if (!c.take(args[1], c.type, q->sizes(), false, &k) || !c.take(args[2], c.type, vs, false, &v) ||
            !c.take(args[5], at::kFloat, {s.H}, true, &a) || !c.take(args[6], c.type, gs, true, &g) ||
            !c.take(args[7], at::kFloat, ss, true, &S0) || !c.take(args[8], at::kInt, {B}, true, &lens) ||
            !to_float(args[9], &scale))
            Py_RETURN_NONE;
        const size_t wsb = lr_decay_attn_workspace_size(B, L, s.H, s.Hk, s.dk, s.dv, c.io);
        if (wsb == 0 || wsb > size_t(INT64_MAX)) Py_RETURN_NONE;
        at::Tensor o, Sf, ws;
        int rc;
        {
            const Unlocked unlocked;
            o = at::empty(vs, q->options());
            Sf = at::empty(ss, q->options().dtype(at::kFloat));
            ws = at::empty({static_cast<int64_t>(wsb)}, q->options().dtype(at::kByte));
            launched = true;
            rc = lr_decay_attn_fwd(q->data_ptr(), k, v, static_cast<float *>(a), g, static_cast<int32_t *>(lens), scale,
                                   static_cast<float *>(S0), o.data_ptr(), Sf.data_ptr<float>(), B, L, s.H, s.Hk, s.dk,
                                   s.dv, c.io, ws.data_ptr(), wsb, c.stream());
        }
        if (rc != LR_OK) return refused(rc);
        const Ref po(THPVariable_Wrap(o)), ps(THPVariable_Wrap(Sf)), pw(THPVariable_Wrap(ws));
        return po.o && ps.o && pw.o ? PyTuple_Pack(3, po.o, ps.o, pw.o) : nullptr;
    } catch (...) {
        return thrown(launched);
    }
}

// (x, G, gamma, beta, z, act code, eps, out) -> y
PyObject *group_norm_act(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 8) Py_RETURN_NONE;
    bool launched = false;
    try {
        Call c;
        const at::Tensor *x = c.first(args[0]);
        int64_t G, act;
        float eps;
        if (x == nullptr || x->dim() < 1 || !to_int(args[1], &G) || !to_int(args[5], &act) ||
            !to_float(args[6], &eps))
            Py_RETURN_NONE;
        const int64_t C = x->size(-1);
        if (G < 1 || C % G != 0) Py_RETURN_NONE;
        void *gamma, *beta, *z, *out;
        if (!c.take(args[2], at::kFloat, {C}, true, &gamma) || !c.take(args[3], at::kFloat, {C}, true, &beta) ||
            !c.take(args[4], c.type, x->sizes(), true, &z) || !c.take(args[7], c.type, x->sizes(), true, &out))
            Py_RETURN_NONE;
        at::Tensor y;
        int rc;
        {
            const Unlocked unlocked;
            if (out == nullptr) {
                y = at::empty(x->sizes(), x->options());
                out = y.data_ptr();
            }
            launched = true;
            rc = lr_group_norm_act(x->data_ptr(), z, static_cast<float *>(gamma), static_cast<float *>(beta), out,
                                   x->numel() / C, C, G, eps, static_cast<lr_act>(act), c.io, c.stream());
        }
        if (rc != LR_OK) return refused(rc);
        return y.defined() ? THPVariable_Wrap(y) : Ref::share(args[7]);
    } catch (...) {
        return thrown(launched);
    }
}

// A pair of results: new tensors, or the caller's own where one was given.
PyObject *pair_of(const at::Tensor &a, const at::Tensor &b, PyObject *given_b) {
    const Ref pa(THPVariable_Wrap(a)), pb(b.defined() ? THPVariable_Wrap(b) : Ref::share(given_b));
    return pa.o && pb.o ? PyTuple_Pack(2, pa.o, pb.o) : nullptr;
}

// (x, w, bias, state, lens, act code) -> (y, state)
PyObject *causal_conv(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 6) Py_RETURN_NONE;
    bool launched = false;
    try {
        Call c;
        const at::Tensor *x = c.first_rows(args[0], 3);
        int64_t act, ldx;
        if (x == nullptr || !THPVariable_CheckExact(args[1]) || !to_int(args[5], &act)) Py_RETURN_NONE;
        const at::Tensor &wt = THPVariable_Unpack(args[1]);
        const int64_t B = x->size(0), L = x->size(1), C = x->size(2), W = wt.dim() == 2 ? wt.size(1) : 0;
        if (W < 2) Py_RETURN_NONE;
        const int64_t ws[] = {C, W}, ss[] = {B, W - 1, C};
        void *px, *w, *bias, *state, *lens;
        if (!c.rows(args[0], false, false, &px, &ldx, x->sizes()) || !c.take(args[1], at::kFloat, ws, false, &w) ||
            !c.take(args[2], at::kFloat, {C}, true, &bias) || !c.take(args[3], c.type, ss, true, &state) ||
            !c.take(args[4], at::kInt, {B}, true, &lens))
            Py_RETURN_NONE;
        at::Tensor y, Sn;
        int rc;
        {
            const Unlocked unlocked;
            y = at::empty(x->sizes(), x->options());
            Sn = at::empty(ss, x->options());
            launched = true;
            rc = lr_causal_conv_fwd(px, ldx, static_cast<float *>(w), static_cast<float *>(bias), state,
                                    static_cast<int32_t *>(lens), y.data_ptr(), Sn.data_ptr(), B, L, C, W,
                                    static_cast<lr_act>(act), c.io, c.stream());
        }
        if (rc != LR_OK) return refused(rc);
        return pair_of(y, Sn, nullptr);
    } catch (...) {
        return thrown(launched);
    }
}

// (x, w, bias, state, state_out, act code) -> (y, state)
PyObject *causal_conv_step(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 6) Py_RETURN_NONE;
    bool launched = false;
    try {
        Call c;
        const at::Tensor *x = c.first_rows(args[0], 2);
        int64_t act, ldx;
        if (x == nullptr || !THPVariable_CheckExact(args[1]) || !to_int(args[5], &act)) Py_RETURN_NONE;
        const at::Tensor &wt = THPVariable_Unpack(args[1]);
        const int64_t B = x->size(0), C = x->size(1), W = wt.dim() == 2 ? wt.size(1) : 0;
        if (W < 2) Py_RETURN_NONE;
        const int64_t ws[] = {C, W}, ss[] = {B, W - 1, C};
        void *px, *w, *bias, *state, *out;
        if (!c.rows(args[0], false, false, &px, &ldx, x->sizes()) || !c.take(args[1], at::kFloat, ws, false, &w) ||
            !c.take(args[2], at::kFloat, {C}, true, &bias) || !c.take(args[3], c.type, ss, true, &state) ||
            !c.take(args[4], c.type, ss, true, &out))
            Py_RETURN_NONE;
        at::Tensor y, Sn;
        int rc;
        {
            const Unlocked unlocked;
            y = at::empty(x->sizes(), x->options());
            if (out == nullptr) {
                Sn = at::empty(ss, x->options());
                out = Sn.data_ptr();
            }
            launched = true;
            rc = lr_causal_conv_step(px, ldx, static_cast<float *>(w), static_cast<float *>(bias), state, out,
                                     y.data_ptr(), B, C, W, static_cast<lr_act>(act), c.io, c.stream());
        }
        if (rc != LR_OK) return refused(rc);
        return pair_of(y, Sn, args[4]);
    } catch (...) {
        return thrown(launched);
    }
}

// What both forms of the selective scan with heads take: (x, dt, Bm, Cm, A_log, H, G, z,
// Dskip, dt_bias, state, ..., softplus)
struct Scan {
    int64_t H, G, P, N, ldx, lddt, ldb, ldc, ldz;
    void *x, *dt, *Bm, *Cm, *z, *A, *skip, *bias, *S;
    // tensors whose rows leave 16-byte boundaries, to be copied: a projection's z does where
    // dt, one column a head, stands beside it
    struct Apart {
        at::Tensor t;
        void **p;
        int64_t *ld;
    };
    std::vector<Apart> apart;
    bool whole_rows(const Call &c, PyObject *o, bool optional, void **p, int64_t *ld, at::IntArrayRef shape) {
        if (c.rows(o, true, optional, p, ld, shape)) return true;
        if (!c.like(o, shape)) return false;
        apart.push_back({THPVariable_Unpack(o), p, ld});
        return true;
    }
    // (with the interpreter released)
    void copy_apart() {
        if (apart.empty()) return;
        const at::NoGradGuard no_grad;
        for (Apart &a : apart) {
            a.t = a.t.clone(at::MemoryFormat::Contiguous);
            *a.p = a.t.data_ptr();
            *a.ld = a.t.size(-1);
        }
    }
    bool of(const Call &c, const at::Tensor &xt, PyObject *const *args) {
        if (!to_int(args[5], &H) || !to_int(args[6], &G) || H < 1 || G < 1 || H % G != 0 || xt.size(-1) % H != 0 ||
            !THPVariable_CheckExact(args[2]))
            return false;
        const at::Tensor &bt = THPVariable_Unpack(args[2]);
        const bool prompt = xt.dim() == 3;
        if (bt.dim() != xt.dim() || bt.size(-1) % G != 0) return false;
        P = xt.size(-1) / H, N = bt.size(-1) / G;
        if (P < 1 || N < 1) return false;
        const int64_t B = xt.size(0), L = prompt ? xt.size(1) : 1;
        const int64_t dt3[] = {B, L, H}, bc3[] = {B, L, G * N}, dt2[] = {B, H}, bc2[] = {B, G * N}, ss[] = {B, H, P, N};
        const at::IntArrayRef ds = prompt ? at::IntArrayRef(dt3) : at::IntArrayRef(dt2);
        const at::IntArrayRef bs = prompt ? at::IntArrayRef(bc3) : at::IntArrayRef(bc2);
        return whole_rows(c, args[0], false, &x, &ldx, xt.sizes()) && c.rows(args[1], false, false, &dt, &lddt, ds) &&
               whole_rows(c, args[2], false, &Bm, &ldb, bs) && whole_rows(c, args[3], false, &Cm, &ldc, bs) &&
               c.take(args[4], at::kFloat, {H}, false, &A) && whole_rows(c, args[7], true, &z, &ldz, xt.sizes()) &&
               c.take(args[8], at::kFloat, {H}, true, &skip) && c.take(args[9], at::kFloat, {H}, true, &bias) &&
               c.take(args[10], at::kFloat, ss, true, &S);
    }
};
float *f32(void *p) { return static_cast<float *>(p); }

// (x, dt, Bm, Cm, A_log, H, G, z, Dskip, dt_bias, S0, lens, softplus) -> (y, S_final, workspace)
PyObject *selective_heads(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 13) Py_RETURN_NONE;
    bool launched = false;
    try {
        Call c;
        Scan s;
        int64_t soft;
        void *lens;
        const at::Tensor *x = c.first_rows(args[0], 3);
        if (x == nullptr || !s.of(c, *x, args) || !to_int(args[12], &soft)) Py_RETURN_NONE;
        const int64_t B = x->size(0), L = x->size(1);
        if (!c.take(args[11], at::kInt, {B}, true, &lens)) Py_RETURN_NONE;
        const size_t wsb = lr_selective_heads_workspace_size(B, L, s.H, s.G, s.P, s.N, c.io);
        if (wsb == 0 || wsb > size_t(INT64_MAX)) Py_RETURN_NONE;
        at::Tensor y, Sf, ws;
        int rc;
        {
            const Unlocked unlocked;
            s.copy_apart();
            y = at::empty(x->sizes(), x->options());
            Sf = at::empty({B, s.H, s.P, s.N}, x->options().dtype(at::kFloat));
            ws = at::empty({static_cast<int64_t>(wsb)}, x->options().dtype(at::kByte));
            launched = true;
            rc = lr_selective_heads_fwd(s.x, s.ldx, s.dt, s.lddt, s.Bm, s.ldb, s.Cm, s.ldc, s.z, s.ldz, f32(s.A),
                                        f32(s.bias), f32(s.skip), static_cast<int32_t *>(lens), f32(s.S), y.data_ptr(),
                                        Sf.data_ptr<float>(), B, L, s.H, s.G, s.P, s.N, c.io, soft != 0, ws.data_ptr(),
                                        wsb, c.stream());
        }
        if (rc != LR_OK) return refused(rc);
        const Ref py(THPVariable_Wrap(y)), ps(THPVariable_Wrap(Sf)), pw(THPVariable_Wrap(ws));
        return py.o && ps.o && pw.o ? PyTuple_Pack(3, py.o, ps.o, pw.o) : nullptr;
    } catch (...) {
        return thrown(launched);
    }
}

// (x, dt, Bm, Cm, A_log, H, G, z, Dskip, dt_bias, S, S_out, softplus) -> (y, S_new)
PyObject *selective_heads_step(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 13) Py_RETURN_NONE;
    bool launched = false;
    try {
        Call c;
        Scan s;
        int64_t soft;
        void *out;
        const at::Tensor *x = c.first_rows(args[0], 2);
        if (x == nullptr || !s.of(c, *x, args) || !to_int(args[12], &soft)) Py_RETURN_NONE;
        const int64_t B = x->size(0), ss[] = {B, s.H, s.P, s.N};
        if (!c.take(args[11], at::kFloat, ss, true, &out)) Py_RETURN_NONE;
        at::Tensor y, Sn;
        int rc;
        {
            const Unlocked unlocked;
            s.copy_apart();
            y = at::empty(x->sizes(), x->options());
            if (out == nullptr) {
                Sn = at::empty(ss, x->options().dtype(at::kFloat));
                out = Sn.data_ptr();
            }
            launched = true;
            rc = lr_selective_heads_step(s.x, s.ldx, s.dt, s.lddt, s.Bm, s.ldb, s.Cm, s.ldc, s.z, s.ldz, f32(s.A),
                                         f32(s.bias), f32(s.skip), f32(s.S), f32(out), y.data_ptr(), B, s.H, s.G, s.P,
                                         s.N, c.io, soft != 0, c.stream());
        }
        if (rc != LR_OK) return refused(rc);
        return pair_of(y, Sn, args[11]);
    } catch (...) {
        return thrown(launched);
    }
}

// (q, k, H, Hk, norm code, gamma_q, gamma_k, freqs, pos, pairs code, eps) -> (q, k)
PyObject *head_norm_rope(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 11) Py_RETURN_NONE;
    bool launched = false;
    try {
        Call c;
        const at::Tensor *q = c.first_rows(args[0], 0);
        int64_t H, Hk, norm, pairs, ldq, ldk, rot = 0;
        float eps;
        if (q == nullptr || !to_int(args[2], &H) || H < 1 || !to_int(args[4], &norm) || !to_int(args[9], &pairs) ||
            !to_float(args[10], &eps) || q->size(-1) % H != 0)
            Py_RETURN_NONE;
        Hk = H;
        if (args[3] != Py_None && (!to_int(args[3], &Hk) || Hk < 1)) Py_RETURN_NONE;
        if (args[1] == Py_None) Hk = 0;
        const int64_t d = q->size(-1) / H;
        std::vector<int64_t> lead(q->sizes().begin(), q->sizes().end() - 1), ks(lead);
        ks.push_back(Hk * d);
        void *pq, *pk, *gq, *gk, *freqs = nullptr, *pos = nullptr;
        if (!c.rows(args[0], false, false, &pq, &ldq, q->sizes()) || !c.rows(args[1], false, true, &pk, &ldk, ks) ||
            !c.take(args[5], at::kFloat, {d}, true, &gq) || !c.take(args[6], at::kFloat, {d}, true, &gk))
            Py_RETURN_NONE;
        if (args[7] != Py_None) {
            if (!THPVariable_CheckExact(args[7])) Py_RETURN_NONE;
            const int64_t m = THPVariable_Unpack(args[7]).numel();
            if (m < 1 || 2 * m > d || !c.take(args[7], at::kFloat, {m}, false, &freqs) ||
                !c.take(args[8], at::kInt, lead, false, &pos))
                Py_RETURN_NONE;
            rot = 2 * m;
        }
        at::Tensor qo, ko;
        int rc;
        {
            const Unlocked unlocked;
            qo = at::empty(q->sizes(), q->options());
            if (Hk > 0) ko = at::empty(ks, q->options());
            launched = true;
            rc = lr_head_norm_rope(pq, ldq, pk, ldk, f32(gq), f32(gk), f32(freqs), static_cast<int32_t *>(pos),
                                   qo.data_ptr(), ko.defined() ? ko.data_ptr() : nullptr, q->numel() / (H * d), H, Hk, d,
                                   rot, static_cast<lr_norm>(norm), eps, static_cast<lr_pairs>(pairs), c.io, c.stream());
        }
        if (rc != LR_OK) return refused(rc);
        return pair_of(qo, ko, Py_None);
    } catch (...) {
        return thrown(launched);
    }
}

template <typename F>
PyCFunction fast(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef kMethods[] = {
    {"decay_attn", fast(decay_attn), METH_FASTCALL, nullptr},
    {"decay_attn_step", fast(decay_attn_step), METH_FASTCALL, nullptr},
    {"group_norm_act", fast(group_norm_act), METH_FASTCALL, nullptr},
    {"causal_conv", fast(causal_conv), METH_FASTCALL, nullptr},
    {"causal_conv_step", fast(causal_conv_step), METH_FASTCALL, nullptr},
    {"selective_heads", fast(selective_heads), METH_FASTCALL, nullptr},
    {"selective_heads_step", fast(selective_heads_step), METH_FASTCALL, nullptr},
    {"head_norm_rope", fast(head_norm_rope), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_lrtorch", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lrtorch() { return PyModule_Create(&kModule); }
