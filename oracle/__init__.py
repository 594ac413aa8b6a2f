"""Float64 CPU oracle for the gated linear-recurrence scans.

TEST INFRASTRUCTURE ONLY.  The oracle is the correctness reference for the
CUDA library in ``selective_state_space_chunked_gb300``.  It shares no code
with that library and never imports it.  Only ``tests/``, the smoke check in
``__graft_entry__`` and the CPU-baseline / reference arm of ``bench.py`` may
import this package; the product path must never route through it.

The arithmetic lives in ``lro_oracle.c`` (plain sequential C over float64,
compiled with ``-O2`` and without ``-ffast-math``).  This module only builds
that file with gcc and marshals numpy arrays to it.

Functions (sources are cited in ``lro_oracle.c``):

* :func:`selective_scan`  -- cortexnet ``MultiScaleSSM._selective_scan`` plus
  the D skip and silu(z) gate of its ``forward``.
* :func:`rglru_scan`      -- lrnnx ``RGLRU.step`` fallback update, every step.
* :func:`hgrn2`           -- HGRN2 Attention ``S_t = diag(g_t) S_{t-1} + v_t k_t^T``
  with the readout ``o_t = S_t q_t``.
* :func:`minmax_scan`     -- minmaxrnc ``MinMaxNeuron`` recurrence
  ``x_t = max(min(r_t, x_{t-1}), s_t)``, every state returned.

* :func:`decay_attn`      -- linear attention with a decay for each head.
* :func:`group_norm_act`  -- group norm per row with an activation and a gate.
* :func:`selective_heads` -- selective scan with heads (by :func:`decay_attn`).
* :func:`causal_conv`     -- short causal convolution, channels last (numpy).
* :func:`head_norm_rope`  -- norm and rotation of heads (numpy).

All are pinned against closed forms, brute force and library routines in
``tests/test_oracle_pins.py``, ``tests/test_decay_oracle_pins.py`` and
``tests/test_layer_oracle_pins.py``.
"""
from __future__ import annotations

import ctypes
import os
import subprocess
import tempfile
import threading

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
_SRC = os.path.join(_HERE, "lro_oracle.c")
_BUILD_DIR = os.path.join(_HERE, "_build")
_LIB_PATH = os.path.join(_BUILD_DIR, "liblro.so")

_lock = threading.Lock()
_lib = None


def build(force: bool = False) -> str:
    """Compile ``lro_oracle.c`` into ``oracle/_build/liblro.so`` with gcc.

    OpenMP is used when the compiler supports it (the loops over independent
    channels / heads are then spread over host cores); the arithmetic inside
    each loop is unchanged.  Returns the path of the shared library.
    """
    if (not force and os.path.exists(_LIB_PATH)
            and os.path.getmtime(_LIB_PATH) >= os.path.getmtime(_SRC)):
        return _LIB_PATH
    os.makedirs(_BUILD_DIR, exist_ok=True)
    fd, tmp = tempfile.mkstemp(suffix=".so", dir=_BUILD_DIR)
    os.close(fd)
    base = ["gcc", "-O2", "-std=c11", "-fPIC", "-shared", "-fno-fast-math",
            "-ffp-contract=off", _SRC, "-o", tmp, "-lm"]
    try:
        try:
            subprocess.run(base[:1] + ["-fopenmp"] + base[1:], check=True,
                           capture_output=True)
        except subprocess.CalledProcessError:
            subprocess.run(base, check=True, capture_output=True)
        os.replace(tmp, _LIB_PATH)
    finally:
        if os.path.exists(tmp):
            os.unlink(tmp)
    return _LIB_PATH


def _load():
    global _lib
    with _lock:
        if _lib is None:
            lib = ctypes.CDLL(build())
            dp = ctypes.POINTER(ctypes.c_double)
            i64 = ctypes.c_int64
            lib.lro_selective_scan_ref.argtypes = [
                dp, dp, dp, dp, dp, dp, dp, dp, ctypes.c_int,
                i64, i64, i64, i64, dp, dp, ctypes.c_int]
            lib.lro_selective_scan_ref.restype = ctypes.c_int
            lib.lro_rglru_scan_ref.argtypes = [
                dp, dp, dp, dp, ctypes.c_double, dp, i64, i64, i64, dp, dp,
                ctypes.c_int]
            lib.lro_rglru_scan_ref.restype = ctypes.c_int
            lib.lro_hgrn2_ref.argtypes = [
                dp, dp, dp, dp, dp, i64, i64, i64, i64, i64, dp, dp,
                ctypes.c_int]
            lib.lro_hgrn2_ref.restype = ctypes.c_int
            lib.lro_minmax_scan_ref.argtypes = [
                dp, dp, dp, i64, i64, i64, dp, dp, ctypes.c_int]
            lib.lro_minmax_scan_ref.restype = ctypes.c_int
            lib.lro_decay_attn_ref.argtypes = [
                dp, dp, dp, dp, dp, ctypes.POINTER(i64), ctypes.c_double, dp, i64, i64, i64, i64, i64,
                i64, dp, dp, ctypes.c_int]
            lib.lro_decay_attn_ref.restype = ctypes.c_int
            lib.lro_group_norm_act_ref.argtypes = [
                dp, dp, dp, dp, i64, i64, i64, ctypes.c_double, ctypes.c_int, dp, ctypes.c_int]
            lib.lro_group_norm_act_ref.restype = ctypes.c_int
            lib.lro_max_threads.argtypes = []
            lib.lro_max_threads.restype = ctypes.c_int
            _lib = lib
    return _lib


def max_threads() -> int:
    """Number of host threads the oracle's parallel loops use by default."""
    return int(_load().lro_max_threads())


def _f64(a):
    """Widen any array-like (numpy or torch, any float dtype) to float64."""
    if a is None:
        return None
    if hasattr(a, "detach"):  # torch tensor: widen exactly, then to numpy
        a = a.detach().to("cpu").double().numpy()
    return np.ascontiguousarray(np.asarray(a, dtype=np.float64))


def _ptr(a):
    if a is None:
        return None
    return a.ctypes.data_as(ctypes.POINTER(ctypes.c_double))


def selective_scan(x, dt, Bm, Cm, A_log, z=None, Dskip=None, h0=None,
                   dt_softplus=True, threads=0):
    """Selective SSM scan in float64.

    x, dt, z: (B, L, D); Bm, Cm: (B, L, N); A_log: (D, N); Dskip: (D,);
    h0: (B, D, N).  Returns ``(y (B, L, D), h_final (B, D, N))`` as float64.
    """
    x, dt, Bm, Cm, A_log = map(_f64, (x, dt, Bm, Cm, A_log))
    z, Dskip, h0 = _f64(z), _f64(Dskip), _f64(h0)
    Bsz, L, D = x.shape
    N = Bm.shape[-1]
    assert dt.shape == x.shape and Bm.shape == (Bsz, L, N) and Cm.shape == (Bsz, L, N)
    assert A_log.shape == (D, N)
    assert z is None or z.shape == x.shape
    assert Dskip is None or Dskip.shape == (D,)
    assert h0 is None or h0.shape == (Bsz, D, N)
    y = np.zeros((Bsz, L, D), dtype=np.float64)
    hf = np.zeros((Bsz, D, N), dtype=np.float64)
    rc = _load().lro_selective_scan_ref(
        _ptr(x), _ptr(dt), _ptr(z), _ptr(Bm), _ptr(Cm), _ptr(A_log),
        _ptr(Dskip), _ptr(h0), int(bool(dt_softplus)), Bsz, L, D, N,
        _ptr(y), _ptr(hf), int(threads))
    if rc != 0:
        raise ValueError("lro_selective_scan_ref rejected its arguments")
    return y, hf


def rglru_scan(x, r, i, a_log, c=8.0, h0=None, threads=0):
    """RG-LRU scan in float64.

    x, r, i: (B, L, D) with r, i already sigmoid-activated; a_log: (D,);
    h0: (B, D).  Returns ``(y (B, L, D), h_final (B, D))`` as float64.
    """
    x, r, i, a_log = map(_f64, (x, r, i, a_log))
    h0 = _f64(h0)
    Bsz, L, D = x.shape
    assert r.shape == x.shape and i.shape == x.shape and a_log.shape == (D,)
    assert h0 is None or h0.shape == (Bsz, D)
    y = np.zeros((Bsz, L, D), dtype=np.float64)
    hf = np.zeros((Bsz, D), dtype=np.float64)
    rc = _load().lro_rglru_scan_ref(
        _ptr(x), _ptr(r), _ptr(i), _ptr(a_log), float(c), _ptr(h0),
        Bsz, L, D, _ptr(y), _ptr(hf), int(threads))
    if rc != 0:
        raise ValueError("lro_rglru_scan_ref rejected its arguments")
    return y, hf


def hgrn2(q, k, v, g, H, S0=None, threads=0):
    """HGRN2 matrix-state recurrence in float64.

    q, k: (B, L, H*dk); v, g: (B, L, H*dv); S0: (B, H, dv, dk).
    Returns ``(o (B, L, H*dv), S_final (B, H, dv, dk))`` as float64.
    """
    q, k, v, g = map(_f64, (q, k, v, g))
    S0 = _f64(S0)
    Bsz, L, HK = q.shape
    HV = v.shape[-1]
    assert HK % H == 0 and HV % H == 0
    dk, dv = HK // H, HV // H
    assert k.shape == q.shape and g.shape == v.shape and v.shape[:2] == (Bsz, L)
    assert S0 is None or S0.shape == (Bsz, H, dv, dk)
    o = np.zeros((Bsz, L, HV), dtype=np.float64)
    Sf = np.zeros((Bsz, H, dv, dk), dtype=np.float64)
    rc = _load().lro_hgrn2_ref(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(S0), Bsz, L, H, dk, dv,
        _ptr(o), _ptr(Sf), int(threads))
    if rc != 0:
        raise ValueError("lro_hgrn2_ref rejected its arguments")
    return o, Sf


def minmax_scan(r, s, x0=None, threads=0):
    """MinMax recurrence x_t = max(min(r_t, x_{t-1}), s_t) in float64.

    r, s: (B, L, D); x0: (B, D) (zero when None).  Returns
    ``(y (B, L, D) = the states after every step, x_final (B, D))``.
    """
    r, s = map(_f64, (r, s))
    x0 = _f64(x0)
    Bsz, L, D = r.shape
    assert s.shape == r.shape and (x0 is None or x0.shape == (Bsz, D))
    y = np.zeros((Bsz, L, D), dtype=np.float64)
    xf = np.zeros((Bsz, D), dtype=np.float64)
    rc = _load().lro_minmax_scan_ref(_ptr(r), _ptr(s), _ptr(x0), Bsz, L, D, _ptr(y), _ptr(xf),
                                     int(threads))
    if rc != 0:
        raise ValueError("lro_minmax_scan_ref rejected its arguments")
    return y, xf


def decay_attn(q, k, v, H, Hk=None, a_log=None, g=None, S0=None, lens=None, scale=1.0, threads=0):
    """Linear attention with a decay for each head in float64.

    q, k: (B, L, Hk*dk); v: (B, L, H*dv); a_log: (H,); g: (B, L, H);
    S0: (B, H, dv, dk); lens: (B,).  Returns ``(o (B, L, H*dv), S_final)``.
    """
    q, k, v = map(_f64, (q, k, v))
    a_log, g, S0 = _f64(a_log), _f64(g), _f64(S0)
    Hk = H if Hk is None else Hk
    Bsz, L, HK = q.shape
    HV = v.shape[-1]
    assert HK % Hk == 0 and HV % H == 0 and H % Hk == 0
    dk, dv = HK // Hk, HV // H
    assert k.shape == q.shape and v.shape[:2] == (Bsz, L)
    assert a_log is None or a_log.shape == (H,)
    assert g is None or g.shape == (Bsz, L, H)
    assert S0 is None or S0.shape == (Bsz, H, dv, dk)
    n = None
    if lens is not None:
        n = np.ascontiguousarray(np.asarray(lens.cpu() if hasattr(lens, "cpu") else lens, dtype=np.int64))
        assert n.shape == (Bsz,)
    o = np.zeros((Bsz, L, HV), dtype=np.float64)
    Sf = np.zeros((Bsz, H, dv, dk), dtype=np.float64)
    rc = _load().lro_decay_attn_ref(
        _ptr(q), _ptr(k), _ptr(v), _ptr(a_log), _ptr(g),
        None if n is None else n.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)), float(scale), _ptr(S0),
        Bsz, L, H, Hk, dk, dv, _ptr(o), _ptr(Sf), int(threads))
    if rc != 0:
        raise ValueError("lro_decay_attn_ref rejected its arguments")
    return o, Sf


def group_norm_act(x, G, gamma=None, beta=None, z=None, act="none", eps=1e-5, threads=0):
    """Group norm of every row of x (N, C) in float64, then the activation
    ("none" or "silu") and the gate silu(z).  Returns y (N, C)."""
    x = _f64(x)
    gamma, beta, z = _f64(gamma), _f64(beta), _f64(z)
    N, C = x.shape
    y = np.zeros((N, C), dtype=np.float64)
    rc = _load().lro_group_norm_act_ref(_ptr(x), _ptr(z), _ptr(gamma), _ptr(beta), N, C, G, float(eps),
                                        int(act == "silu"), _ptr(y), int(threads))
    if rc != 0:
        raise ValueError("lro_group_norm_act_ref rejected its arguments")
    return y


def _silu(x):
    with np.errstate(over="ignore"):   # e^-x past float64's range: the quotient is 0
        return x / (1.0 + np.exp(-x))


def _lengths(lens, Bsz, L):
    if lens is None:
        return [L] * Bsz
    return [min(max(int(n), 0), L) for n in lens]


def selective_heads(x, dt, Bm, Cm, A_log, H, G=1, z=None, Dskip=None, dt_bias=None, S0=None, lens=None,
                    dt_softplus=True, threads=0):
    """Selective scan with heads in float64: S = exp(-exp(A_log) delta) S + delta x B^T,
    y = (S C + Dskip x) silu(z), delta = softplus(dt + dt_bias).

    x, z: (B, L, H*P); dt: (B, L, H); Bm, Cm: (B, L, G*N); A_log, Dskip, dt_bias: (H,);
    S0: (B, H, P, N); lens: (B,).  Returns ``(y (B, L, H*P), S_final)``.
    """
    x, dt, Bm, Cm, A_log, z, Dskip, dt_bias = map(_f64, (x, dt, Bm, Cm, A_log, z, Dskip, dt_bias))
    Bsz, L, HP = x.shape
    delta = dt if dt_bias is None else dt + dt_bias
    if dt_softplus:
        delta = np.logaddexp(delta, 0.0)
    xh = x.reshape(Bsz, L, H, HP // H)
    y, Sf = decay_attn(Cm, Bm, (delta[..., None] * xh).reshape(x.shape), H, Hk=G, g=-np.exp(A_log) * delta, S0=S0,
                       lens=lens, threads=threads)
    if Dskip is not None:
        y = y + (Dskip[:, None] * xh).reshape(x.shape)
    if z is not None:
        y = y * _silu(z)
    for b, n in enumerate(_lengths(lens, Bsz, L)):
        y[b, n:] = 0.0
    return y, Sf


def causal_conv(x, w, bias=None, state=None, lens=None, act="silu"):
    """Short causal convolution in float64.  x: (B, L, C); w: (C, W); bias: (C,);
    state: (B, W-1, C); lens: (B,).  Returns ``(y (B, L, C), state (B, W-1, C))``."""
    x, w, bias, state = map(_f64, (x, w, bias, state))
    Bsz, L, C = x.shape
    W = w.shape[1]
    y, new = np.zeros((Bsz, L, C)), np.zeros((Bsz, W - 1, C))
    for b, n in enumerate(_lengths(lens, Bsz, L)):
        v = np.concatenate([np.zeros((W - 1, C)) if state is None else state[b], x[b, :n]])
        acc = np.zeros((n, C)) + (0.0 if bias is None else bias)
        for j in range(W):
            acc += w[:, j] * v[j:j + n]
        y[b, :n] = _silu(acc) if act == "silu" else acc
        new[b] = v[n:]
    return y, new


def head_norm_rope(x, H, norm="rms", gamma=None, freqs=None, pos=None, pairs="halves", eps=1e-6):
    """Norm and rotation of the heads of x (..., H*d) in float64 (one of q and k)."""
    x, gamma, freqs, pos = map(_f64, (x, gamma, freqs, pos))
    v = x.reshape(*x.shape[:-1], H, -1).copy()
    if norm != "none":
        s = (v * v).mean(-1, keepdims=True) if norm == "rms" else (v * v).sum(-1, keepdims=True)
        v = v / np.sqrt(s + eps)
    if gamma is not None:
        v = v * gamma
    if freqs is not None:
        m = len(freqs)
        a, b = (slice(0, m), slice(m, 2 * m)) if pairs == "halves" else (slice(0, 2 * m, 2), slice(1, 2 * m, 2))
        p = (pos[..., None] * freqs)[..., None, :]
        v[..., a], v[..., b] = v[..., a] * np.cos(p) - v[..., b] * np.sin(p), v[..., b] * np.cos(p) + v[..., a] * np.sin(p)
    return v.reshape(x.shape)
