// lr_torch.cpp -- the short path of the torch helpers that are called once per
// layer and token, where the GPU's own time is a few microseconds: argument
// checks, result allocation and the call of the C ABI without the interpreter
// between them (host time of a step 16 -> 3.6 us, of a prompt 21 -> 6.9, of a group norm
// 12 -> 3.6).
//
// Each function takes what its helper in binding.py takes and returns what it
// returns, or None where an argument is not already what the kernels take
// (another type or device, not contiguous, shapes that do not match, empty) or
// the call's own checks refused it; nothing has been launched then, and the helper
// goes on to its own checks and conversions, which convert the argument or say what
// is wrong.  Any other status comes back as an int, for the helper to raise: part of
// the call may have run, and it may have updated a state in place.  The interpreter
// is released for the allocations and the call: both may wait for the GPU.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

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

template <typename F>
PyCFunction fast(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef kMethods[] = {
    {"decay_attn", fast(decay_attn), METH_FASTCALL, nullptr},
    {"decay_attn_step", fast(decay_attn_step), METH_FASTCALL, nullptr},
    {"group_norm_act", fast(group_norm_act), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_lrtorch", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lrtorch() { return PyModule_Create(&kModule); }
