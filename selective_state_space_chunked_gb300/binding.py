"""ctypes binding of ``liblrscan.so`` (the C ABI in ``include/lrscan.h``).

Two layers, both argument marshalling only -- every step of every scan runs
in the library's CUDA kernels:

* ``lr_*`` functions with the C names and signatures (pointers as ints);
* torch conveniences (:func:`selective_scan`, :func:`rglru_scan`,
  :func:`hgrn2`, :func:`decay_attn`, ...) that check shapes and dtypes, allocate outputs and the
  workspace with torch, pass the current CUDA stream and raise
  :class:`LrError` on a non-zero status.  Given host tensors they copy the
  inputs to the current CUDA device and the outputs back (the end-to-end
  path); given device tensors they stay on the device.

There is no fallback: if the library is missing this module raises at import (the
extension module with the helpers' short path may be missing; a warning says so).
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import threading
import warnings
from typing import Optional, Tuple

import torch

from . import build as _build

LR_F32, LR_BF16 = 0, 1
LR_OK = 0
LR_ERR_INVALID_ARG, LR_ERR_UNSUPPORTED, LR_ERR_MISALIGNED = -1, -2, -3
LR_ERR_WORKSPACE, LR_ERR_CUDA, LR_ERR_TIMEOUT, LR_ERR_RANGE = -4, -5, -6, -7
LR_ACT_NONE, LR_ACT_SILU = 0, 1
LR_NORM_NONE, LR_NORM_RMS, LR_NORM_L2 = 0, 1, 2
LR_PAIRS_HALVES, LR_PAIRS_NEIGHBOURS = 0, 1

_IO = {torch.float32: LR_F32, torch.bfloat16: LR_BF16}

# (name, restype, argtypes) of every exported C symbol
_P, _I64, _F, _I, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int, ctypes.c_size_t
SIGNATURES = {
    "lr_status_string": (ctypes.c_char_p, [_I]),
    "lr_version": (_I, []),
    "lr_check_status": (_I, [_P, _P]),
    "lr_set_split_override": (_I, [_I]),
    "lr_test_withhold_split": (_I, [_I, _I]),
    "lr_set_host_chunk_steps": (_I64, [_I64]),
    "lr_set_selective_warmup": (_I64, [_I64]),
    "lr_selective_scan_workspace_size": (_SZ, [_I64, _I64, _I64, _I64, _I]),
    "lr_selective_scan_fwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                   _I64, _I64, _I64, _I64, _I, _I, _P, _SZ, _P]),
    "lr_rglru_scan_workspace_size": (_SZ, [_I64, _I64, _I64, _I]),
    "lr_rglru_scan_fwd": (_I, [_P, _P, _P, _P, _F, _P, _P, _P,
                               _I64, _I64, _I64, _I, _P, _SZ, _P]),
    "lr_rglru_scan_fwd_noalloc": (_I, [_P, _P, _P, _P, _F, _P, _P, _P,
                                       _I64, _I64, _I64, _I, _P]),
    "lr_hgrn2_workspace_size": (_SZ, [_I64, _I64, _I64, _I64, _I64, _I]),
    "lr_hgrn2_fwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64,
                          _I64, _I64, _I, _P, _SZ, _P]),
    "lr_rglru_scan_preact_fwd": (_I, [_P, _P, _P, _P, _F, _P, _P, _P,
                                      _I64, _I64, _I64, _I, _P, _SZ, _P]),
    "lr_hgrn2_preact_fwd": (_I, [_P, _P, _P, _P, _F, _P, _P, _P, _I64, _I64, _I64, _I64,
                                 _I64, _I64, _I, _P, _SZ, _P]),
    "lr_minmax_scan_workspace_size": (_SZ, [_I64, _I64, _I64, _I]),
    "lr_minmax_scan_fwd": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _SZ, _P]),
    "lr_selective_scan_step": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                    _I64, _I64, _I64, _I, _I, _P]),
    "lr_rglru_scan_step": (_I, [_P, _P, _P, _P, _F, _P, _P, _P, _I64, _I64, _I, _P]),
    "lr_hgrn2_step": (_I, [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I, _P]),
    "lr_minmax_scan_step": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I, _P]),
    "lr_selective_scan_fwd_host_workspace_size": (_SZ, [_I64, _I64, _I64, _I64, _I]),
    "lr_selective_scan_fwd_host": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                        _I64, _I64, _I64, _I64, _I, _I, _P, _SZ, _P]),
    "lr_rglru_scan_fwd_host_workspace_size": (_SZ, [_I64, _I64, _I64, _I]),
    "lr_rglru_scan_fwd_host": (_I, [_P, _P, _P, _P, _F, _P, _P, _P,
                                    _I64, _I64, _I64, _I, _P, _SZ, _P]),
    "lr_hgrn2_fwd_host_workspace_size": (_SZ, [_I64, _I64, _I64, _I64, _I64, _I]),
    "lr_hgrn2_fwd_host": (_I, [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64,
                               _I64, _I64, _I, _P, _SZ, _P]),
    "lr_minmax_scan_fwd_host_workspace_size": (_SZ, [_I64, _I64, _I64, _I]),
    "lr_minmax_scan_fwd_host": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _SZ, _P]),
    "lr_selective_scan_fwd_host_async": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                              _I64, _I64, _I64, _I64, _I, _I, _P, _SZ, _P]),
    "lr_rglru_scan_fwd_host_async": (_I, [_P, _P, _P, _P, _F, _P, _P, _P,
                                          _I64, _I64, _I64, _I, _P, _SZ, _P]),
    "lr_hgrn2_fwd_host_async": (_I, [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64,
                                     _I64, _I64, _I, _P, _SZ, _P]),
    "lr_minmax_scan_fwd_host_async": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _SZ, _P]),
    "lr_host_sync": (_I, []),
    "lr_decay_attn_workspace_size": (_SZ, [_I64, _I64, _I64, _I64, _I64, _I64, _I]),
    "lr_decay_attn_fwd": (_I, [_P, _P, _P, _P, _P, _P, _F, _P, _P, _P, _I64, _I64, _I64, _I64, _I64,
                               _I64, _I, _P, _SZ, _P]),
    "lr_decay_attn_step": (_I, [_P, _P, _P, _P, _P, _F, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _I,
                                _P]),
    "lr_decay_attn_fwd_host_workspace_size": (_SZ, [_I64, _I64, _I64, _I64, _I64, _I64, _I]),
    "lr_decay_attn_fwd_host": (_I, [_P, _P, _P, _P, _P, _F, _P, _P, _P, _I64, _I64, _I64, _I64, _I64,
                                    _I64, _I, _P, _SZ, _P]),
    "lr_decay_attn_fwd_host_async": (_I, [_P, _P, _P, _P, _P, _F, _P, _P, _P, _I64, _I64, _I64, _I64,
                                          _I64, _I64, _I, _P, _SZ, _P]),
    "lr_group_norm_act": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _F, _I, _I, _P]),
    "lr_selective_heads_workspace_size": (_SZ, [_I64, _I64, _I64, _I64, _I64, _I64, _I]),
    "lr_selective_heads_fwd": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _P, _P, _P,
                                    _I64, _I64, _I64, _I64, _I64, _I64, _I, _I, _P, _SZ, _P]),
    "lr_selective_heads_step": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _P, _P,
                                     _I64, _I64, _I64, _I64, _I64, _I, _I, _P]),
    "lr_causal_conv_fwd": (_I, [_P, _I64, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I, _I, _P]),
    "lr_causal_conv_step": (_I, [_P, _I64, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _P]),
    "lr_head_norm_rope": (_I, [_P, _I64, _P, _I64, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _I, _F,
                               _I, _I, _P]),
}


def _load():
    path = _build.LIB_PATH
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with selective_state_space_chunked_gb300."
            "build.build() (nvcc, sm_103a). There is no CPU fallback.")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()
LIB_PATH = _build.LIB_PATH


class _NoTorchModule:
    """In the place of an extension module that cannot be loaded: declines every
    call, so that the helpers take their own path."""

    @staticmethod
    def _decline(*args):
        return None

    decay_attn = decay_attn_step = group_norm_act = _decline
    causal_conv = causal_conv_step = selective_heads = selective_heads_step = head_norm_rope = _decline


def _load_torch_module():
    try:
        if not _build.torch_module_matches():
            raise ImportError("missing, or built against another torch")
        spec = importlib.util.spec_from_file_location("_lrtorch", _build.TORCH_MODULE)
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        return mod
    except (ImportError, OSError) as e:
        warnings.warn(f"{_build.TORCH_MODULE} cannot be used ({e}): calls of one token take longer; build it with "
                      "selective_state_space_chunked_gb300.build.build()", RuntimeWarning)
        return _NoTorchModule()


# The helpers that run once per layer and token first offer their arguments to
# this module, which takes those that are already what the kernels take and
# answers None to the others (a status, where a call failed past its checks).
_lrtorch = _load_torch_module()


class LrError(RuntimeError):
    """A non-zero lrscan status."""

    def __init__(self, code: int, where: str = ""):
        self.code = int(code)
        msg = lr_status_string(code)
        super().__init__(f"{where}: {msg}" if where else msg)


# ---------------------------------------------------------------- C names
def lr_status_string(code: int) -> str:
    return _lib.lr_status_string(int(code)).decode()


def lr_version() -> int:
    return int(_lib.lr_version())


def lr_check_status(workspace, stream: int = 0) -> int:
    """Status of the latest call that used ``workspace`` (a device pointer;
    None = the built-in scratch of lr_rglru_scan_fwd_noalloc); synchronises
    ``stream`` and resets the status."""
    return int(_lib.lr_check_status(workspace or None, stream or None))


def lr_set_split_override(splits: int) -> int:
    return int(_lib.lr_set_split_override(int(splits)))


def lr_set_host_chunk_steps(steps: int) -> int:
    """Chunk length of the host-buffer path (0 = automatic); returns the previous."""
    return int(_lib.lr_set_host_chunk_steps(int(steps)))


def lr_set_selective_warmup(max_steps: int) -> int:
    """Longest warm-up of the selective scan's pieces in steps (0 = carries
    by look-back only, negative = automatic: 2048 for bf16 I/O, 0 for fp32);
    returns the previous setting (-1 = automatic)."""
    return int(_lib.lr_set_selective_warmup(int(max_steps)))


def lr_test_withhold_split(split: int, timeout_ms: int = 1000) -> int:
    return int(_lib.lr_test_withhold_split(int(split), int(timeout_ms)))


def lr_selective_scan_workspace_size(B, L, D, N, io) -> int:
    return int(_lib.lr_selective_scan_workspace_size(B, L, D, N, io))


def lr_selective_scan_fwd(x, dt, z, Bm, Cm, A_log, Dskip, h0, y, h_final,
                          B, L, D, N, io, dt_softplus, workspace, ws_bytes,
                          stream) -> int:
    return int(_lib.lr_selective_scan_fwd(x, dt, z, Bm, Cm, A_log, Dskip, h0, y,
                                          h_final, B, L, D, N, io, dt_softplus,
                                          workspace, ws_bytes, stream))


def lr_rglru_scan_workspace_size(B, L, D, io) -> int:
    return int(_lib.lr_rglru_scan_workspace_size(B, L, D, io))


def lr_rglru_scan_fwd(x, r, i, a_log, c, h0, y, h_final, B, L, D, io,
                      workspace, ws_bytes, stream) -> int:
    return int(_lib.lr_rglru_scan_fwd(x, r, i, a_log, c, h0, y, h_final, B, L, D,
                                      io, workspace, ws_bytes, stream))


def lr_rglru_scan_fwd_noalloc(x, r, i, a_log, c, h0, y, h_final, B, L, D, io,
                              stream) -> int:
    """RG-LRU scan using the library's built-in scratch (no workspace)."""
    return int(_lib.lr_rglru_scan_fwd_noalloc(x, r, i, a_log, c, h0, y, h_final, B, L,
                                              D, io, stream))


def lr_hgrn2_workspace_size(B, L, H, dk, dv, io) -> int:
    return int(_lib.lr_hgrn2_workspace_size(B, L, H, dk, dv, io))


def lr_hgrn2_fwd(q, k, v, g, S0, o, S_final, B, L, H, dk, dv, chunk, io,
                 workspace, ws_bytes, stream) -> int:
    return int(_lib.lr_hgrn2_fwd(q, k, v, g, S0, o, S_final, B, L, H, dk, dv,
                                 chunk, io, workspace, ws_bytes, stream))


def lr_rglru_scan_preact_fwd(x, r_pre, i_pre, a_log, c, h0, y, h_final, B, L, D, io,
                             workspace, ws_bytes, stream) -> int:
    return int(_lib.lr_rglru_scan_preact_fwd(x, r_pre, i_pre, a_log, c, h0, y, h_final, B, L, D,
                                             io, workspace, ws_bytes, stream))


def lr_hgrn2_preact_fwd(q, k, v, f, lb, S0, o, S_final, B, L, H, dk, dv, chunk, io,
                        workspace, ws_bytes, stream) -> int:
    return int(_lib.lr_hgrn2_preact_fwd(q, k, v, f, lb, S0, o, S_final, B, L, H, dk, dv, chunk,
                                        io, workspace, ws_bytes, stream))


def lr_minmax_scan_workspace_size(B, L, D, io) -> int:
    return int(_lib.lr_minmax_scan_workspace_size(B, L, D, io))


def lr_minmax_scan_fwd(r, s, x0, y, x_final, B, L, D, io, workspace, ws_bytes, stream) -> int:
    return int(_lib.lr_minmax_scan_fwd(r, s, x0, y, x_final, B, L, D, io, workspace, ws_bytes,
                                       stream))


def lr_selective_scan_step(x, dt, z, Bm, Cm, A_log, Dskip, h_in, h_out, y, B, D, N,
                           io, dt_softplus, stream) -> int:
    return int(_lib.lr_selective_scan_step(x, dt, z, Bm, Cm, A_log, Dskip, h_in, h_out,
                                           y, B, D, N, io, dt_softplus, stream))


def lr_rglru_scan_step(x, r, i, a_log, c, h_in, h_out, y, B, D, io, stream) -> int:
    return int(_lib.lr_rglru_scan_step(x, r, i, a_log, c, h_in, h_out, y, B, D, io,
                                       stream))


def lr_minmax_scan_step(r, s, x_in, x_out, y, B, D, io, stream) -> int:
    return int(_lib.lr_minmax_scan_step(r, s, x_in, x_out, y, B, D, io, stream))


def lr_hgrn2_step(q, k, v, g, S_in, S_out, o, B, H, dk, dv, io, stream) -> int:
    return int(_lib.lr_hgrn2_step(q, k, v, g, S_in, S_out, o, B, H, dk, dv, io,
                                  stream))


def lr_selective_scan_fwd_host_workspace_size(B, L, D, N, io) -> int:
    return int(_lib.lr_selective_scan_fwd_host_workspace_size(B, L, D, N, io))


def lr_selective_scan_fwd_host(x, dt, z, Bm, Cm, A_log, Dskip, h0, y, h_final, B, L, D, N, io,
                               dt_softplus, workspace, ws_bytes, stream) -> int:
    """Selective scan on host buffers (device workspace only)."""
    return int(_lib.lr_selective_scan_fwd_host(x, dt, z, Bm, Cm, A_log, Dskip, h0, y, h_final,
                                               B, L, D, N, io, dt_softplus, workspace, ws_bytes,
                                               stream))


def lr_rglru_scan_fwd_host_workspace_size(B, L, D, io) -> int:
    return int(_lib.lr_rglru_scan_fwd_host_workspace_size(B, L, D, io))


def lr_rglru_scan_fwd_host(x, r, i, a_log, c, h0, y, h_final, B, L, D, io, workspace, ws_bytes,
                           stream) -> int:
    """RG-LRU scan on host buffers (device workspace only)."""
    return int(_lib.lr_rglru_scan_fwd_host(x, r, i, a_log, c, h0, y, h_final, B, L, D, io,
                                           workspace, ws_bytes, stream))


def lr_hgrn2_fwd_host_workspace_size(B, L, H, dk, dv, io) -> int:
    return int(_lib.lr_hgrn2_fwd_host_workspace_size(B, L, H, dk, dv, io))


def lr_hgrn2_fwd_host(q, k, v, g, S0, o, S_final, B, L, H, dk, dv, chunk, io, workspace, ws_bytes,
                      stream) -> int:
    """HGRN2 on host buffers (device workspace only)."""
    return int(_lib.lr_hgrn2_fwd_host(q, k, v, g, S0, o, S_final, B, L, H, dk, dv, chunk, io,
                                      workspace, ws_bytes, stream))


def lr_minmax_scan_fwd_host_workspace_size(B, L, D, io) -> int:
    return int(_lib.lr_minmax_scan_fwd_host_workspace_size(B, L, D, io))


def lr_minmax_scan_fwd_host(r, s, x0, y, x_final, B, L, D, io, workspace, ws_bytes, stream) -> int:
    """MinMax scan on host buffers (device workspace only)."""
    return int(_lib.lr_minmax_scan_fwd_host(r, s, x0, y, x_final, B, L, D, io, workspace, ws_bytes,
                                            stream))


def lr_selective_scan_fwd_host_async(x, dt, z, Bm, Cm, A_log, Dskip, h0, y, h_final, B, L, D, N, io,
                                     dt_softplus, workspace, ws_bytes, stream) -> int:
    """As lr_selective_scan_fwd_host, returning once the work is queued."""
    return int(_lib.lr_selective_scan_fwd_host_async(x, dt, z, Bm, Cm, A_log, Dskip, h0, y, h_final,
                                                     B, L, D, N, io, dt_softplus, workspace, ws_bytes,
                                                     stream))


def lr_rglru_scan_fwd_host_async(x, r, i, a_log, c, h0, y, h_final, B, L, D, io, workspace, ws_bytes,
                                 stream) -> int:
    """As lr_rglru_scan_fwd_host, returning once the work is queued."""
    return int(_lib.lr_rglru_scan_fwd_host_async(x, r, i, a_log, c, h0, y, h_final, B, L, D, io,
                                                 workspace, ws_bytes, stream))


def lr_hgrn2_fwd_host_async(q, k, v, g, S0, o, S_final, B, L, H, dk, dv, chunk, io, workspace, ws_bytes,
                            stream) -> int:
    """As lr_hgrn2_fwd_host, returning once the work is queued."""
    return int(_lib.lr_hgrn2_fwd_host_async(q, k, v, g, S0, o, S_final, B, L, H, dk, dv, chunk, io,
                                            workspace, ws_bytes, stream))


def lr_minmax_scan_fwd_host_async(r, s, x0, y, x_final, B, L, D, io, workspace, ws_bytes, stream) -> int:
    """As lr_minmax_scan_fwd_host, returning once the work is queued."""
    return int(_lib.lr_minmax_scan_fwd_host_async(r, s, x0, y, x_final, B, L, D, io, workspace, ws_bytes,
                                                  stream))


def lr_host_sync() -> int:
    """Waits for every host-buffer call queued on the current device."""
    return int(_lib.lr_host_sync())


def lr_decay_attn_workspace_size(B, L, H, Hk, dk, dv, io) -> int:
    return int(_lib.lr_decay_attn_workspace_size(B, L, H, Hk, dk, dv, io))


def lr_decay_attn_fwd(q, k, v, a_log, g, lens, scale, S0, o, S_final, B, L, H, Hk, dk, dv, io,
                      workspace, ws_bytes, stream) -> int:
    return _lib.lr_decay_attn_fwd(q, k, v, a_log, g, lens, scale, S0, o, S_final, B, L, H, Hk, dk, dv,
                                  io, workspace, ws_bytes, stream)


def lr_decay_attn_step(q, k, v, a_log, g, scale, S_in, S_out, o, B, H, Hk, dk, dv, io, stream) -> int:
    return _lib.lr_decay_attn_step(q, k, v, a_log, g, scale, S_in, S_out, o, B, H, Hk, dk, dv, io,
                                   stream)


def lr_decay_attn_fwd_host_workspace_size(B, L, H, Hk, dk, dv, io) -> int:
    return int(_lib.lr_decay_attn_fwd_host_workspace_size(B, L, H, Hk, dk, dv, io))


def lr_decay_attn_fwd_host(q, k, v, a_log, g, scale, S0, o, S_final, B, L, H, Hk, dk, dv, io, workspace,
                           ws_bytes, stream) -> int:
    """Decayed linear attention on host buffers (device workspace only)."""
    return int(_lib.lr_decay_attn_fwd_host(q, k, v, a_log, g, scale, S0, o, S_final, B, L, H, Hk, dk, dv,
                                           io, workspace, ws_bytes, stream))


def lr_decay_attn_fwd_host_async(q, k, v, a_log, g, scale, S0, o, S_final, B, L, H, Hk, dk, dv, io,
                                 workspace, ws_bytes, stream) -> int:
    """As lr_decay_attn_fwd_host, returning once the work is queued."""
    return int(_lib.lr_decay_attn_fwd_host_async(q, k, v, a_log, g, scale, S0, o, S_final, B, L, H, Hk,
                                                 dk, dv, io, workspace, ws_bytes, stream))


def lr_group_norm_act(x, z, gamma, beta, y, N, C, G, eps, act, io, stream) -> int:
    return _lib.lr_group_norm_act(x, z, gamma, beta, y, N, C, G, eps, act, io, stream)


def lr_selective_heads_workspace_size(B, L, H, G, P, N, io) -> int:
    return int(_lib.lr_selective_heads_workspace_size(B, L, H, G, P, N, io))


def lr_selective_heads_fwd(x, ldx, dt, lddt, Bm, ldb, Cm, ldc, z, ldz, A_log, dt_bias, Dskip, lens, S0, y, S_final,
                           B, L, H, G, P, N, io, dt_softplus, workspace, ws_bytes, stream) -> int:
    return _lib.lr_selective_heads_fwd(x, ldx, dt, lddt, Bm, ldb, Cm, ldc, z, ldz, A_log, dt_bias, Dskip, lens, S0, y,
                                       S_final, B, L, H, G, P, N, io, dt_softplus, workspace, ws_bytes, stream)


def lr_selective_heads_step(x, ldx, dt, lddt, Bm, ldb, Cm, ldc, z, ldz, A_log, dt_bias, Dskip, S_in, S_out, y, B, H, G,
                            P, N, io, dt_softplus, stream) -> int:
    return _lib.lr_selective_heads_step(x, ldx, dt, lddt, Bm, ldb, Cm, ldc, z, ldz, A_log, dt_bias, Dskip, S_in, S_out,
                                        y, B, H, G, P, N, io, dt_softplus, stream)


def lr_causal_conv_fwd(x, ldx, w, bias, state, lens, y, state_out, B, L, C, W, act, io, stream) -> int:
    return _lib.lr_causal_conv_fwd(x, ldx, w, bias, state, lens, y, state_out, B, L, C, W, act, io, stream)


def lr_causal_conv_step(x, ldx, w, bias, state_in, state_out, y, B, C, W, act, io, stream) -> int:
    return _lib.lr_causal_conv_step(x, ldx, w, bias, state_in, state_out, y, B, C, W, act, io, stream)


def lr_head_norm_rope(q, ldq, k, ldk, gamma_q, gamma_k, freqs, pos, q_out, k_out, N, H, Hk, d, rot, norm, eps, pairs,
                      io, stream) -> int:
    return _lib.lr_head_norm_rope(q, ldq, k, ldk, gamma_q, gamma_k, freqs, pos, q_out, k_out, N, H, Hk, d, rot, norm,
                                  eps, pairs, io, stream)


# ------------------------------------------------------------ torch helpers
def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _aligned(t: torch.Tensor) -> torch.Tensor:
    """t, contiguous, from a 16-byte boundary: a contiguous view starts anywhere
    (a step of one row, a row of an odd width, a layer of stacked parameters)."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _dev(t: Optional[torch.Tensor], device) -> Optional[torch.Tensor]:
    if t is None:
        return None
    if t.device != device:   # (of another GPU too: its memory is not the kernels' to read)
        t = t.to(device, non_blocking=True)
    return _aligned(t)


def _check(rc: int, where: str):
    if rc != LR_OK:
        _tls.ws = None   # a call that failed on the host recorded no device status
        raise LrError(rc, where)


def _io_of(t: torch.Tensor) -> int:
    if t.dtype not in _IO:
        raise TypeError(f"unsupported I/O dtype {t.dtype}; use float32 or bfloat16")
    return _IO[t.dtype]


def _same(ref: torch.Tensor, *ts):
    for t in ts:
        if t is not None and t.dtype != ref.dtype:
            raise TypeError("all activation tensors must share one dtype")


# The workspace of this thread's latest call through the torch helpers: its
# first bytes hold that call's device-side status (see status()).
_tls = threading.local()


def last_workspace() -> Optional[torch.Tensor]:
    """Workspace tensor of this thread's latest call through a torch helper."""
    return getattr(_tls, "ws", None)


def _workspace(nbytes: int, device, given: Optional[torch.Tensor]):
    if nbytes == (1 << 64) - 1:
        raise LrError(LR_ERR_CUDA, "workspace size query")
    if nbytes == 0:
        _tls.ws = None
        return None, 0
    if given is not None:
        ws, n = given, given.numel() * given.element_size()
    else:
        ws, n = torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes
    _tls.ws = ws
    return ws, n


def _target_device(*ts):
    for t in ts:
        if t is not None and t.device.type == "cuda":
            return t.device
    return torch.device("cuda", torch.cuda.current_device())


def _back(out: torch.Tensor, host: bool) -> torch.Tensor:
    if not host:
        return out
    h = torch.empty(out.shape, dtype=out.dtype, pin_memory=True)
    h.copy_(out, non_blocking=True)
    return h


def _outputs(out, specs, dev):
    """Device buffers the kernel writes, and the caller's host destinations.

    ``out`` is None or a tuple of tensors matching ``specs`` (shape, dtype):
    all on the GPU (the kernel writes them in place) or all on the host
    (results are copied into them; pinned memory keeps the copy
    asynchronous and avoids allocating a pinned buffer per call)."""
    if out is None:
        return [torch.empty(sh, dtype=dt, device=dev) for sh, dt in specs], None
    if len(out) != len(specs):
        raise ValueError(f"out must hold {len(specs)} tensors")
    for o, (sh, dt) in zip(out, specs):
        if tuple(o.shape) != tuple(sh) or o.dtype != dt or not o.is_contiguous():
            raise ValueError(f"out tensor {tuple(o.shape)} {o.dtype} does not match "
                             f"{tuple(sh)} {dt} (contiguous)")
    on_gpu = [o.device.type == "cuda" for o in out]
    if all(on_gpu):
        if any(o.device != dev for o in out):
            raise ValueError("out tensors must be on the inputs' GPU")
        return list(out), None
    if any(on_gpu):
        raise ValueError("out tensors must be all on the GPU or all on the host")
    return [torch.empty(sh, dtype=dt, device=dev) for sh, dt in specs], list(out)


# ---- host buffers: the library's chunked host path (lr_*_fwd_host)
_HOST_WS = {}


def _host_route(acts, out) -> bool:
    """True when every activation and every given result tensor is in host
    memory: the call then goes to the library's host-buffer entry point."""
    if any(t is not None and t.device.type == "cuda" for t in acts):
        return False
    return out is None or all(o.device.type != "cuda" for o in out)


def _h(t: Optional[torch.Tensor], dtype=None) -> Optional[torch.Tensor]:
    if t is None:
        return None
    if t.device.type == "cuda":
        t = t.cpu()
    if dtype is not None:
        t = t.to(dtype)
    return _aligned(t)


def _host_outputs(out, specs):
    """Host result tensors: the caller's, or new pinned ones."""
    if out is None:
        return [torch.empty(sh, dtype=dt, pin_memory=True) for sh, dt in specs]
    if len(out) != len(specs):
        raise ValueError(f"out must hold {len(specs)} tensors")
    for o, (sh, dt) in zip(out, specs):
        if tuple(o.shape) != tuple(sh) or o.dtype != dt or not o.is_contiguous():
            raise ValueError(f"out tensor {tuple(o.shape)} {o.dtype} does not match "
                             f"{tuple(sh)} {dt} (contiguous)")
    return list(out)


def _host_workspace(nbytes: int, given: Optional[torch.Tensor]):
    """Device staging for a host-buffer call: the caller's tensor, or one
    kept per device and grown as needed."""
    if nbytes == (1 << 64) - 1:
        raise LrError(LR_ERR_CUDA, "workspace size query")
    if nbytes == 0:
        return None, 0
    if given is not None:
        _tls.ws = given
        return given, given.numel() * given.element_size()
    dev = torch.cuda.current_device()
    ws = _HOST_WS.get(dev)
    if ws is None or ws.numel() < nbytes:
        _HOST_WS.pop(dev, None)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", dev))
        _HOST_WS[dev] = ws
    _tls.ws = ws
    return ws, nbytes


# tensors that host-buffer calls queued with sync_host=False still read or
# write (inputs, results, workspaces), per device, until host_sync()
_ASYNC_KEEP = {}


def _async_workspace(nbytes: int, given: Optional[torch.Tensor]):
    """Device staging for a queued host-buffer call: the caller's tensor, or a
    new one (calls in flight must not share one)."""
    if nbytes == (1 << 64) - 1:
        raise LrError(LR_ERR_CUDA, "workspace size query")
    if nbytes == 0:
        return None, 0
    if given is not None:
        _tls.ws = given
        return given, given.numel() * given.element_size()
    ws = torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", torch.cuda.current_device()))
    _tls.ws = ws
    return ws, nbytes


def _host_entry(sync_fn, async_fn, nbytes, workspace, sync_host: bool, keep):
    """The host-buffer entry point and its workspace: synchronous, or queued
    (its tensors kept alive until host_sync())."""
    if sync_host:
        ws, wsb = _host_workspace(nbytes, workspace)
        return sync_fn, ws, wsb
    ws, wsb = _async_workspace(nbytes, workspace)
    _ASYNC_KEEP.setdefault(torch.cuda.current_device(), []).extend(
        [t for t in list(keep) + [ws] if t is not None])
    return async_fn, ws, wsb


def host_sync() -> None:
    """Waits for every host-buffer call queued with ``sync_host=False`` on the
    current device; their results are then in host memory (read each call's
    device-side status afterwards with ``status(workspace)``)."""
    _check(lr_host_sync(), "lr_host_sync")
    _ASYNC_KEEP.pop(torch.cuda.current_device(), None)


def _host_stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _finish(bufs, host_out, host: bool, dev, sync_host: bool):
    if host_out is not None:
        for dst, src in zip(host_out, bufs):
            dst.copy_(src, non_blocking=True)
        res = host_out
    else:
        res = [_back(b, host) for b in bufs]
    if (host or host_out is not None) and sync_host:
        torch.cuda.current_stream(dev).synchronize()
    return tuple(res)


def selective_scan(x, dt, Bm, Cm, A_log, z=None, Dskip=None, h0=None,
                   dt_softplus: bool = True, workspace=None, out=None,
                   sync_host: bool = True) -> Tuple[torch.Tensor, torch.Tensor]:
    """Selective SSM scan.  x, dt, z: (B, L, D); Bm, Cm: (B, L, 16), all one
    dtype (float32 or bfloat16); A_log: (D, 16) fp32; Dskip: (D,) fp32;
    h0: (B, D, 16) fp32.  Returns (y (B, L, D) in the I/O dtype, h_final
    (B, D, 16) fp32); ``out=(y, h_final)`` gives the result tensors (GPU or
    host).  Host inputs with host (or no) ``out`` run the library's
    host-buffer path (chunked, copies overlapping the scan; pinned memory
    keeps the copies asynchronous); ``workspace`` is then its device
    staging buffer.  With ``sync_host=False`` a host-buffer call returns once
    its work is queued, so consecutive calls overlap; ``host_sync()`` waits
    for it (each queued call without a ``workspace`` gets a new one)."""
    if _host_route((x, dt, z, Bm, Cm), out):
        x, dt, z, Bm, Cm = (_h(t) for t in (x, dt, z, Bm, Cm))
        A_log, Dskip, h0 = (_h(t, torch.float32) for t in (A_log, Dskip, h0))
        _same(x, dt, z, Bm, Cm)
        io = _io_of(x)
        B, L, D = x.shape
        N = Bm.shape[-1]
        y, hf = _host_outputs(out, [((B, L, D), x.dtype), ((B, D, N), torch.float32)])
        fn, ws, wsb = _host_entry(lr_selective_scan_fwd_host, lr_selective_scan_fwd_host_async,
                                  lr_selective_scan_fwd_host_workspace_size(B, L, D, N, io), workspace,
                                  sync_host, (x, dt, z, Bm, Cm, A_log, Dskip, h0, y, hf))
        _check(fn(_ptr(x), _ptr(dt), _ptr(z), _ptr(Bm), _ptr(Cm), _ptr(A_log), _ptr(Dskip), _ptr(h0),
                  _ptr(y), _ptr(hf), B, L, D, N, io, int(bool(dt_softplus)), _ptr(ws), wsb,
                  _host_stream()), fn.__name__)
        return y, hf
    host = x.device.type != "cuda"
    dev = _target_device(x)
    x, dt, z, Bm, Cm = (_dev(t, dev) for t in (x, dt, z, Bm, Cm))
    A_log, Dskip, h0 = (_dev(None if t is None else t.float(), dev) for t in (A_log, Dskip, h0))
    _same(x, dt, z, Bm, Cm)
    io = _io_of(x)
    B, L, D = x.shape
    N = Bm.shape[-1]
    (y, hf), host_out = _outputs(out, [((B, L, D), x.dtype), ((B, D, N), torch.float32)], dev)
    ws, wsb = _workspace(lr_selective_scan_workspace_size(B, L, D, N, io), dev, workspace)
    stream = torch.cuda.current_stream(dev).cuda_stream
    _check(lr_selective_scan_fwd(_ptr(x), _ptr(dt), _ptr(z), _ptr(Bm), _ptr(Cm),
                                 _ptr(A_log), _ptr(Dskip), _ptr(h0), _ptr(y),
                                 _ptr(hf), B, L, D, N, io, int(bool(dt_softplus)),
                                 _ptr(ws), wsb, stream), "lr_selective_scan_fwd")
    return _finish((y, hf), host_out, host, dev, sync_host)


def rglru_scan(x, r, i, a_log, c: float = 8.0, h0=None, workspace=None, out=None,
               sync_host: bool = True, gates_preact: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """RG-LRU scan.  x, r, i: (B, L, D) (r, i after their sigmoid, or before
    it with ``gates_preact=True``: the kernel applies it), one dtype;
    a_log: (D,) fp32; h0: (B, D) fp32.  Returns (y (B, L, D), h_final (B, D)
    fp32); ``out=(y, h_final)`` gives the result tensors (GPU or host).  Host
    inputs with host (or no) ``out`` run the library's host-buffer path
    (activated gates only; ``sync_host=False`` queues it, as for
    ``selective_scan``)."""
    if not gates_preact and _host_route((x, r, i), out):
        x, r, i = (_h(t) for t in (x, r, i))
        a_log, h0 = (_h(t, torch.float32) for t in (a_log, h0))
        _same(x, r, i)
        io = _io_of(x)
        B, L, D = x.shape
        y, hf = _host_outputs(out, [((B, L, D), x.dtype), ((B, D), torch.float32)])
        fn, ws, wsb = _host_entry(lr_rglru_scan_fwd_host, lr_rglru_scan_fwd_host_async,
                                  lr_rglru_scan_fwd_host_workspace_size(B, L, D, io), workspace, sync_host,
                                  (x, r, i, a_log, h0, y, hf))
        _check(fn(_ptr(x), _ptr(r), _ptr(i), _ptr(a_log), float(c), _ptr(h0), _ptr(y), _ptr(hf),
                  B, L, D, io, _ptr(ws), wsb, _host_stream()), fn.__name__)
        return y, hf
    host = x.device.type != "cuda"
    dev = _target_device(x)
    x, r, i = (_dev(t, dev) for t in (x, r, i))
    a_log, h0 = (_dev(None if t is None else t.float(), dev) for t in (a_log, h0))
    _same(x, r, i)
    io = _io_of(x)
    B, L, D = x.shape
    (y, hf), host_out = _outputs(out, [((B, L, D), x.dtype), ((B, D), torch.float32)], dev)
    ws, wsb = _workspace(lr_rglru_scan_workspace_size(B, L, D, io), dev, workspace)
    stream = torch.cuda.current_stream(dev).cuda_stream
    fwd = lr_rglru_scan_preact_fwd if gates_preact else lr_rglru_scan_fwd
    _check(fwd(_ptr(x), _ptr(r), _ptr(i), _ptr(a_log), float(c), _ptr(h0), _ptr(y), _ptr(hf),
               B, L, D, io, _ptr(ws), wsb, stream), fwd.__name__)
    return _finish((y, hf), host_out, host, dev, sync_host)


def hgrn2(q, k, v, g, H: int, S0=None, chunk: int = 64, workspace=None, out=None,
          sync_host: bool = True, gate_lb: Optional[float] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """HGRN2 matrix-state recurrence.  q, k: (B, L, H*dk); v, g: (B, L, H*dv)
    (g after its activation and lower bound; with ``gate_lb`` set, g is the
    pre-activation f and the kernel forms lb + (1 - lb) sigmoid(f)), one
    dtype (bfloat16 or float32); S0: (B, H, dv, dk) fp32.  Returns (o (B, L, H*dv), S_final
    (B, H, dv, dk) fp32); ``out=(o, S_final)`` gives the result tensors (GPU
    or host).  Host inputs with host (or no) ``out`` run the library's
    host-buffer path (activated gates only; ``sync_host=False`` queues it, as
    for ``selective_scan``).  Raises ValueError when the hidden size is not
    divisible by the head count."""
    if q.shape[-1] % H or v.shape[-1] % H:
        raise ValueError(f"hidden size {q.shape[-1]} is not divisible by {H} heads")
    if gate_lb is None and _host_route((q, k, v, g), out):
        q, k, v, g = (_h(t) for t in (q, k, v, g))
        S0 = _h(S0, torch.float32)
        _same(q, k, v, g)
        io = _io_of(q)
        B, L, HK = q.shape
        dk, dv = HK // H, v.shape[-1] // H
        o, Sf = _host_outputs(out, [((B, L, H * dv), q.dtype), ((B, H, dv, dk), torch.float32)])
        fn, ws, wsb = _host_entry(lr_hgrn2_fwd_host, lr_hgrn2_fwd_host_async,
                                  lr_hgrn2_fwd_host_workspace_size(B, L, H, dk, dv, io), workspace, sync_host,
                                  (q, k, v, g, S0, o, Sf))
        _check(fn(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(S0), _ptr(o), _ptr(Sf),
                  B, L, H, dk, dv, chunk, io, _ptr(ws), wsb, _host_stream()), fn.__name__)
        return o, Sf
    host = q.device.type != "cuda"
    dev = _target_device(q)
    q, k, v, g = (_dev(t, dev) for t in (q, k, v, g))
    S0 = _dev(None if S0 is None else S0.float(), dev)
    _same(q, k, v, g)
    io = _io_of(q)
    B, L, HK = q.shape
    dk, dv = HK // H, v.shape[-1] // H
    (o, Sf), host_out = _outputs(out, [((B, L, H * dv), q.dtype), ((B, H, dv, dk), torch.float32)],
                                 dev)
    ws, wsb = _workspace(lr_hgrn2_workspace_size(B, L, H, dk, dv, io), dev, workspace)
    stream = torch.cuda.current_stream(dev).cuda_stream
    if gate_lb is None:
        _check(lr_hgrn2_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(S0), _ptr(o),
                            _ptr(Sf), B, L, H, dk, dv, chunk, io, _ptr(ws), wsb,
                            stream), "lr_hgrn2_fwd")
    else:
        _check(lr_hgrn2_preact_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), float(gate_lb), _ptr(S0),
                                   _ptr(o), _ptr(Sf), B, L, H, dk, dv, chunk, io, _ptr(ws), wsb,
                                   stream), "lr_hgrn2_preact_fwd")
    return _finish((o, Sf), host_out, host, dev, sync_host)


def minmax_scan(r, s, x0=None, workspace=None, out=None,
                sync_host: bool = True) -> Tuple[torch.Tensor, torch.Tensor]:
    """MinMax recurrence x_t = max(min(r_t, x_{t-1}), s_t).  r, s: (B, L, D),
    one dtype (float32 or bfloat16); x0: (B, D) fp32 or None (zero).
    Returns (y (B, L, D) = the state after every step, x_final (B, D) fp32);
    ``out=(y, x_final)`` gives the result tensors (GPU or host).  Host inputs
    with host (or no) ``out`` run the library's host-buffer path
    (``sync_host=False`` queues it, as for ``selective_scan``)."""
    if _host_route((r, s), out):
        r, s = (_h(t) for t in (r, s))
        x0 = _h(x0, torch.float32)
        _same(r, s)
        io = _io_of(r)
        B, L, D = r.shape
        y, xf = _host_outputs(out, [((B, L, D), r.dtype), ((B, D), torch.float32)])
        fn, ws, wsb = _host_entry(lr_minmax_scan_fwd_host, lr_minmax_scan_fwd_host_async,
                                  lr_minmax_scan_fwd_host_workspace_size(B, L, D, io), workspace, sync_host,
                                  (r, s, x0, y, xf))
        _check(fn(_ptr(r), _ptr(s), _ptr(x0), _ptr(y), _ptr(xf), B, L, D, io, _ptr(ws), wsb,
                  _host_stream()), fn.__name__)
        return y, xf
    host = r.device.type != "cuda"
    dev = _target_device(r)
    r, s = (_dev(t, dev) for t in (r, s))
    x0 = _dev(None if x0 is None else x0.float(), dev)
    _same(r, s)
    io = _io_of(r)
    B, L, D = r.shape
    (y, xf), host_out = _outputs(out, [((B, L, D), r.dtype), ((B, D), torch.float32)], dev)
    ws, wsb = _workspace(lr_minmax_scan_workspace_size(B, L, D, io), dev, workspace)
    stream = torch.cuda.current_stream(dev).cuda_stream
    _check(lr_minmax_scan_fwd(_ptr(r), _ptr(s), _ptr(x0), _ptr(y), _ptr(xf), B, L, D, io, _ptr(ws),
                              wsb, stream), "lr_minmax_scan_fwd")
    return _finish((y, xf), host_out, host, dev, sync_host)


def _heads_of(q, k, v, g, H: int, Hk: Optional[int], ndim: int):
    """(shape of q, Hk, dk, dv, I/O type) of q, k (..., Hk*dk), v (..., H*dv)
    and g (..., H) or None."""
    Hk = H if Hk is None else Hk
    if H < 1 or Hk < 1 or H % Hk:
        raise ValueError(f"{H} value heads cannot share {Hk} key heads")
    qs, vs = q.shape, v.shape
    if len(qs) != ndim or k.shape != qs or len(vs) != ndim or vs[:-1] != qs[:-1]:
        raise ValueError(f"q {tuple(qs)}, k {tuple(k.shape)}, v {tuple(vs)} do not match")
    if qs[-1] % Hk or vs[-1] % H:
        raise ValueError(f"widths {qs[-1]} and {vs[-1]} are not divisible by {Hk} key heads and {H} value heads")
    if g is not None and g.shape != (*qs[:-1], H):
        raise ValueError(f"g must have shape {(*qs[:-1], H)}, not {tuple(g.shape)}")
    dt = q.dtype
    if k.dtype != dt or v.dtype != dt or (g is not None and g.dtype != dt):
        raise TypeError("all activation tensors must share one dtype")
    return qs, Hk, qs[-1] // Hk, vs[-1] // H, _io_of(q)


def _shaped(t: Optional[torch.Tensor], shape, name: str):
    if t is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")


def _stream_of(t: torch.Tensor) -> int:
    """The current stream of t's GPU (a cudaStream_t as an int)."""
    return torch.cuda.current_stream(t.device).cuda_stream


def _act(t: Optional[torch.Tensor], dev) -> Optional[torch.Tensor]:
    """t on the GPU, contiguous and aligned."""
    if t is None or (t.device == dev and t.is_contiguous() and t.data_ptr() % 16 == 0):
        return t
    return _dev(t, dev)


def _par(t: Optional[torch.Tensor], dev) -> Optional[torch.Tensor]:
    """As _act, in float32 (parameters and states)."""
    if t is None or (t.dtype is torch.float32 and t.device == dev and t.is_contiguous() and t.data_ptr() % 16 == 0):
        return t
    return _dev(t.float(), dev)


def _lens_of(lens: Optional[torch.Tensor], L: int, dev):
    """lens as the kernels read them: clamped before they are narrowed, and in 64 bits, since
    L need not fit a narrower type."""
    if lens is None:
        return None
    return _act(lens if lens.dtype is torch.int32 else lens.to(torch.int64).clamp(0, L).to(torch.int32), dev)


def decay_attn(q, k, v, H: int, Hk: Optional[int] = None, a_log=None, g=None, S0=None, lens=None,
               scale: float = 1.0, workspace=None, out=None,
               sync_host: bool = True) -> Tuple[torch.Tensor, torch.Tensor]:
    """Causal linear attention with a decay for each head:
    S_t = exp(a_log[h] + g[b, t, h]) S_{t-1} + v_t k_t^T, o_t = scale S_t q_t.

    q, k: (B, L, Hk*dk); v: (B, L, H*dv); g: (B, L, H) or None, one dtype
    (bfloat16 or float32); a_log: (H,) fp32 or None; ``Hk`` key heads (default
    H), each shared by H/Hk value heads; S0: (B, H, dv, dk) fp32 or None;
    lens: (B,) integers or None: row b has lens[b] steps (its later outputs are
    0 and its state stays).  Returns (o (B, L, H*dv), S_final (B, H, dv, dk)
    fp32); ``out=(o, S_final)`` gives the result tensors (GPU or host).  Host
    inputs with host (or no) ``out`` run the library's host-buffer path (without
    ``lens``; ``sync_host=False`` queues it, as for ``selective_scan``).  A log
    decay above 0 sets LR_ERR_RANGE (see ``check_status``)."""
    if workspace is None and out is None:
        r = _lrtorch.decay_attn(q, k, v, H, Hk, a_log, g, S0, lens, scale)
        if type(r) is tuple:
            o, Sf, _tls.ws = r
            return o, Sf
        if r is not None:
            _check(r, "lr_decay_attn_fwd")
    (B, L, _), Hk, dk, dv, io = _heads_of(q, k, v, g, H, Hk, 3)
    if a_log is not None:
        _shaped(a_log, (H,), "a_log")
    if S0 is not None:
        _shaped(S0, (B, H, dv, dk), "S0")
    if lens is not None:
        _shaped(lens, (B,), "lens")
    specs = (((B, L, H * dv), q.dtype), ((B, H, dv, dk), torch.float32))
    if lens is None and not q.is_cuda and _host_route((q, k, v, g), out):
        q, k, v, g = (_h(t) for t in (q, k, v, g))
        a_log, S0 = (_h(t, torch.float32) for t in (a_log, S0))
        o, Sf = _host_outputs(out, specs)
        fn, ws, wsb = _host_entry(lr_decay_attn_fwd_host, lr_decay_attn_fwd_host_async,
                                  lr_decay_attn_fwd_host_workspace_size(B, L, H, Hk, dk, dv, io), workspace,
                                  sync_host, (q, k, v, a_log, g, S0, o, Sf))
        _check(fn(_ptr(q), _ptr(k), _ptr(v), _ptr(a_log), _ptr(g), float(scale), _ptr(S0), _ptr(o), _ptr(Sf),
                  B, L, H, Hk, dk, dv, io, _ptr(ws), wsb, _host_stream()), fn.__name__)
        return o, Sf
    host = not q.is_cuda
    dev = _target_device(q)
    q, k, v, g = _act(q, dev), _act(k, dev), _act(v, dev), _act(g, dev)
    a_log, S0 = _par(a_log, dev), _par(S0, dev)
    lens = _lens_of(lens, L, dev)
    host_out = None
    if out is None:
        o = torch.empty((B, L, H * dv), dtype=q.dtype, device=dev)
        Sf = torch.empty((B, H, dv, dk), dtype=torch.float32, device=dev)
    else:
        (o, Sf), host_out = _outputs(out, specs, dev)
    ws, wsb = _workspace(lr_decay_attn_workspace_size(B, L, H, Hk, dk, dv, io), dev, workspace)
    rc = _lib.lr_decay_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(a_log), _ptr(g), _ptr(lens), scale,
                                _ptr(S0), o.data_ptr(), Sf.data_ptr(), B, L, H, Hk, dk, dv, io, ws.data_ptr(), wsb,
                                _stream_of(q))
    if rc != LR_OK:
        _check(rc, "lr_decay_attn_fwd")
    if host or host_out is not None:
        return _finish((o, Sf), host_out, host, dev, sync_host)
    return o, Sf


def group_norm_act(x, G: int, gamma=None, beta=None, z=None, act: str = "none", eps: float = 1e-5,
                   out=None) -> torch.Tensor:
    """Group norm of every row of x (..., C) on the GPU in G groups of
    neighbouring channels, then gamma, beta ((C,) fp32 or None), the activation
    ("none" or "silu") and the gate silu(z) (z like x, or None).  Statistics are
    per row.  ``out`` gives the result tensor (x or z itself is allowed)."""
    a = _ACT.get(act)
    if a is None:
        raise ValueError(f"unknown activation {act!r}; use one of {sorted(_ACT)}")
    y = _lrtorch.group_norm_act(x, G, gamma, beta, z, a, eps, out)
    if type(y) is int:
        _check(y, "lr_group_norm_act")
    if y is not None:
        return y
    shape = x.shape
    C = shape[-1]
    if G < 1 or C % G:
        raise ValueError(f"{C} channels cannot be split into {G} groups")
    io = _io_of(x)
    if z is not None:
        _shaped(z, shape, "z")
        _same(x, z)
    if gamma is not None:
        _shaped(gamma, (C,), "gamma")
    if beta is not None:
        _shaped(beta, (C,), "beta")
    dev = x.device if x.is_cuda else _target_device(x)
    x, z, gamma, beta = _act(x, dev), _act(z, dev), _par(gamma, dev), _par(beta, dev)
    if out is None:
        out = torch.empty_like(x)
    elif out.shape != shape or out.dtype != x.dtype or out.device != dev or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {x.dtype} GPU tensor of shape {tuple(shape)}")
    rc = _lib.lr_group_norm_act(x.data_ptr(), _ptr(z), _ptr(gamma), _ptr(beta), out.data_ptr(),
                                x.numel() // C if C else 0, C, G, eps, a, io, _stream_of(x))
    if rc != LR_OK:
        _check(rc, "lr_group_norm_act")
    return out


_ACT = {"none": LR_ACT_NONE, "silu": LR_ACT_SILU}


def _rows(t: Optional[torch.Tensor], dev, whole: bool = False):
    """(t on the GPU, elements between its rows) for t (..., C) whose rows lie evenly
    apart, as the slices of a projection's output do; a copy where they do not, or
    where t does not start on a 16-byte boundary (``whole``: its rows too, unless dense)."""
    if t is None:
        return None, 0
    if t.device != dev:
        t = t.to(dev, non_blocking=True)
    C = t.shape[-1]
    ld, size = None, 1
    for n, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):   # rows from the last axis on
        if n == 1:
            continue
        if ld is None:
            ld = st
        elif st != ld * size:
            ld = -1
        size *= n
    if ld is None:
        ld = C
    if t.numel() == 0 or (C > 1 and t.stride(-1) != 1) or ld < C or t.data_ptr() % 16 or (
            whole and ld != C and ld * t.element_size() % 16):
        return _aligned(t), C
    return t, ld


def _integers(t: Optional[torch.Tensor], shape, name: str):
    _shaped(t, shape, name)
    if t is not None and (t.is_floating_point() or t.dtype is torch.bool):
        raise TypeError(f"{name} must be integers")




def _out_like(out: Optional[torch.Tensor], shape, dtype, dev, name: str = "out"):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if out.shape != torch.Size(shape) or out.dtype != dtype or out.device != dev or not out.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} GPU tensor of shape {tuple(shape)}")
    return out


def _heads_args(x, dt, Bm, Cm, A_log, H: int, G: int, z, Dskip, dt_bias, S, ndim: int):
    """(leading shape, P, N, I/O type) of a selective scan with heads."""
    if H < 1 or G < 1 or H % G:
        raise ValueError(f"{H} heads cannot share {G} groups of B and C")
    lead = x.shape[:-1]
    if x.dim() != ndim or x.shape[-1] == 0 or x.shape[-1] % H:
        raise ValueError(f"x {tuple(x.shape)} does not hold {H} heads")
    if Bm.shape[:-1] != lead or Cm.shape != Bm.shape or Bm.shape[-1] == 0 or Bm.shape[-1] % G:
        raise ValueError(f"x {tuple(x.shape)}, Bm {tuple(Bm.shape)}, Cm {tuple(Cm.shape)} do not match")
    P, N = x.shape[-1] // H, Bm.shape[-1] // G
    _shaped(dt, (*lead, H), "dt")
    _shaped(z, x.shape, "z")
    _shaped(A_log, (H,), "A_log")
    _shaped(dt_bias, (H,), "dt_bias")
    _shaped(Dskip, (H,), "Dskip")
    _shaped(S, (x.shape[0], H, P, N), "the state")
    _same(x, dt, Bm, Cm, z)
    return lead, P, N, _io_of(x)


def selective_heads(x, dt, Bm, Cm, A_log, H: int, G: int = 1, z=None, Dskip=None, dt_bias=None, S0=None, lens=None,
                    dt_softplus: bool = True, workspace=None, out=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Selective scan with heads: S_t = exp(-exp(A_log) delta_t) S_{t-1} + delta_t x_t B_t^T,
    y_t = (S_t C_t + Dskip x_t) silu(z_t), delta = softplus(dt + dt_bias).

    x, z: (B, L, H*P); dt: (B, L, H); Bm, Cm: (B, L, G*N), on the GPU, one dtype (bfloat16
    or float32); slices of wider tensors are read where they stand if their rows keep to
    16-byte boundaries.  A_log, Dskip, dt_bias: (H,) fp32; ``G`` groups of B and C, each
    shared by H/G heads; S0: (B, H, P, N) fp32 or None; lens: (B,) integers or None: row b
    has lens[b] steps (its later outputs are 0 and its state stays); ``dt_softplus=False``:
    delta = dt + dt_bias, at least 0.  z, Dskip, dt_bias may be None.  Returns (y
    (B, L, H*P), S_final (B, H, P, N) fp32); ``out=(y, S_final)`` gives the result tensors.
    A negative or NaN step size sets LR_ERR_RANGE (see ``check_status``)."""
    if workspace is None and out is None:
        r = _lrtorch.selective_heads(x, dt, Bm, Cm, A_log, H, G, z, Dskip, dt_bias, S0, lens, bool(dt_softplus))
        if type(r) is tuple:
            y, S, _tls.ws = r
            return y, S
        if r is not None:
            _check(r, "lr_selective_heads_fwd")
    (B, L), P, N, io = _heads_args(x, dt, Bm, Cm, A_log, H, G, z, Dskip, dt_bias, S0, 3)
    _integers(lens, (B,), "lens")
    dev = _target_device(x)
    y, S = out if out is not None else (None, None)
    with torch.cuda.device(dev):
        x, ldx = _rows(x, dev, True)
        dt, lddt = _rows(dt, dev)
        Bm, ldb = _rows(Bm, dev, True)
        Cm, ldc = _rows(Cm, dev, True)
        z, ldz = _rows(z, dev, True)
        lens = _lens_of(lens, L, dev)
        A_log, Dskip, dt_bias, S0 = (_par(t, dev) for t in (A_log, Dskip, dt_bias, S0))
        y = _out_like(y, (B, L, H * P), x.dtype, dev)
        S = _out_like(S, (B, H, P, N), torch.float32, dev)
        ws, wsb = _workspace(lr_selective_heads_workspace_size(B, L, H, G, P, N, io), dev, workspace)
        _check(lr_selective_heads_fwd(_ptr(x), ldx, _ptr(dt), lddt, _ptr(Bm), ldb, _ptr(Cm), ldc, _ptr(z), ldz,
                                      _ptr(A_log), _ptr(dt_bias), _ptr(Dskip), _ptr(lens), _ptr(S0), _ptr(y), _ptr(S),
                                      B, L, H, G, P, N, io, int(bool(dt_softplus)), _ptr(ws), wsb, _stream_of(x)),
               "lr_selective_heads_fwd")
    return y, S


def selective_heads_step(x, dt, Bm, Cm, A_log, H: int, G: int = 1, z=None, Dskip=None, dt_bias=None, S=None,
                         S_out=None, dt_softplus: bool = True) -> Tuple[torch.Tensor, torch.Tensor]:
    """One token of ``selective_heads``.  x, z: (B, H*P); dt: (B, H); Bm, Cm: (B, G*N); S:
    (B, H, P, N) fp32 or None (zero).  Returns (y (B, H*P), S_new); ``S_out`` gives the
    buffer S_new is written to (it may be ``S`` itself)."""
    r = _lrtorch.selective_heads_step(x, dt, Bm, Cm, A_log, H, G, z, Dskip, dt_bias, S, S_out, bool(dt_softplus))
    if type(r) is tuple:
        return r
    if r is not None:
        _check(r, "lr_selective_heads_step")
    (B,), P, N, io = _heads_args(x, dt, Bm, Cm, A_log, H, G, z, Dskip, dt_bias, S, 2)
    dev = _target_device(x)
    with torch.cuda.device(dev):
        x, ldx = _rows(x, dev, True)
        dt, lddt = _rows(dt, dev)
        Bm, ldb = _rows(Bm, dev, True)
        Cm, ldc = _rows(Cm, dev, True)
        z, ldz = _rows(z, dev, True)
        A_log, Dskip, dt_bias, S = (_par(t, dev) for t in (A_log, Dskip, dt_bias, S))
        S_out = _out_like(S_out, (B, H, P, N), torch.float32, dev, "S_out")
        y = torch.empty((B, H * P), dtype=x.dtype, device=dev)
        _check(lr_selective_heads_step(_ptr(x), ldx, _ptr(dt), lddt, _ptr(Bm), ldb, _ptr(Cm), ldc, _ptr(z), ldz,
                                       _ptr(A_log), _ptr(dt_bias), _ptr(Dskip), _ptr(S), _ptr(S_out), _ptr(y), B, H, G,
                                       P, N, io, int(bool(dt_softplus)), _stream_of(x)), "lr_selective_heads_step")
    return y, S_out


def _conv_args(x, w, bias, state, act: str, ndim: int):
    a = _ACT.get(act)
    if a is None:
        raise ValueError(f"unknown activation {act!r}; use one of {sorted(_ACT)}")
    if x.dim() != ndim or w.dim() != 2 or w.shape[0] != x.shape[-1]:
        raise ValueError(f"x {tuple(x.shape)} and w {tuple(w.shape)} do not match")
    C, W = w.shape
    if bias is not None:
        _shaped(bias, (C,), "bias")
    if state is not None:
        _shaped(state, (x.shape[0], W - 1, C), "state")
        _same(x, state)
    return a, C, W, _io_of(x)


def causal_conv(x, w, bias=None, state=None, lens=None, act: str = "silu",
                out=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Short causal convolution of every channel:
    y_t = act(bias + sum_j w[:, j] x_{t - W + 1 + j}).

    x: (B, L, C) on the GPU, float32 or bfloat16 (a slice of a wider tensor is read
    where it stands); w: (C, W) and bias: (C,) fp32, 2 <= W <= 4; state: (B, W-1, C) in
    x's dtype, the inputs before the first step, oldest first, or None (zeros); lens:
    (B,) integers or None: row b has lens[b] steps (its later outputs are 0); ``act``:
    "silu" or "none".  Returns (y (B, L, C), the state after each row's last step);
    ``out=(y, state)`` gives the result tensors (the state may be ``state`` itself)."""
    if out is None:
        r = _lrtorch.causal_conv(x, w, bias, state, lens, _ACT.get(act))
        if type(r) is tuple:
            return r
        if r is not None:
            _check(r, "lr_causal_conv_fwd")
    a, C, W, io = _conv_args(x, w, bias, state, act, 3)
    B, L, _ = x.shape
    _integers(lens, (B,), "lens")
    dev = _target_device(x)
    y, new = out if out is not None else (None, None)
    with torch.cuda.device(dev):
        x, ldx = _rows(x, dev)
        lens = _lens_of(lens, L, dev)
        w, bias, state = _par(w, dev), _par(bias, dev), _act(state, dev)
        y = _out_like(y, (B, L, C), x.dtype, dev)
        new = _out_like(new, (B, W - 1, C), x.dtype, dev)
        _check(lr_causal_conv_fwd(_ptr(x), ldx, _ptr(w), _ptr(bias), _ptr(state), _ptr(lens), _ptr(y), _ptr(new),
                                  B, L, C, W, a, io, _stream_of(x)), "lr_causal_conv_fwd")
    return y, new


def causal_conv_step(x, w, bias=None, state=None, state_out=None,
                     act: str = "silu") -> Tuple[torch.Tensor, torch.Tensor]:
    """One token of ``causal_conv``.  x: (B, C); state: (B, W-1, C) or None (zeros).
    Returns (y (B, C), the new state); ``state_out`` gives the buffer that it is
    written to (it may be ``state`` itself)."""
    r = _lrtorch.causal_conv_step(x, w, bias, state, state_out, _ACT.get(act))
    if type(r) is tuple:
        return r
    if r is not None:
        _check(r, "lr_causal_conv_step")
    a, C, W, io = _conv_args(x, w, bias, state, act, 2)
    B = x.shape[0]
    dev = _target_device(x)
    with torch.cuda.device(dev):
        x, ldx = _rows(x, dev)
        w, bias, state = _par(w, dev), _par(bias, dev), _act(state, dev)
        new = _out_like(state_out, (B, W - 1, C), x.dtype, dev, "state_out")
        y = torch.empty((B, C), dtype=x.dtype, device=dev)
        _check(lr_causal_conv_step(_ptr(x), ldx, _ptr(w), _ptr(bias), _ptr(state), _ptr(new), _ptr(y), B, C, W, a, io,
                                   _stream_of(x)), "lr_causal_conv_step")
    return y, new


_NORM = {"none": LR_NORM_NONE, "rms": LR_NORM_RMS, "l2": LR_NORM_L2}
_PAIRS = {"halves": LR_PAIRS_HALVES, "neighbours": LR_PAIRS_NEIGHBOURS}


def head_norm_rope(q, k, H: int, Hk: Optional[int] = None, norm: str = "rms", gamma_q=None, gamma_k=None, freqs=None,
                   pos=None, pairs: str = "halves", eps: float = 1e-6, out=None):
    """Norm of every head of q and k, and the rotation of its pairs by the token's
    position, in one pass.

    q: (..., H*d), k: (..., Hk*d) or None, on the GPU, one dtype (bfloat16 or float32;
    slices of a wider tensor are read where they stand); ``Hk``: key heads (default H);
    ``norm``: "rms" (x / sqrt(mean(x^2) + eps)), "l2" (the sum of the squares) or "none";
    gamma_q, gamma_k: (d,) fp32 factors after it, or None; freqs: (rot/2,) fp32, radians
    a position, or None (no rotation): the first rot values of a head are rotated, their
    ``pairs`` being values i and i + rot/2 ("halves") or 2i and 2i + 1 ("neighbours");
    pos: (...) integers within int32.  Returns (q, k) as new dense tensors; ``out`` gives
    them (dense inputs themselves are allowed)."""
    n, p = _NORM.get(norm), _PAIRS.get(pairs)
    if out is None:
        r = _lrtorch.head_norm_rope(q, k, H, Hk, n, gamma_q, gamma_k, freqs, pos, p, eps)
        if type(r) is tuple:
            return r
        if r is not None:
            _check(r, "lr_head_norm_rope")
    if n is None or p is None:
        raise ValueError(f"unknown norm {norm!r} or pairs {pairs!r}; use one of {sorted(_NORM)} and {sorted(_PAIRS)}")
    lead, Hk = q.shape[:-1], 0 if k is None else H if Hk is None else Hk
    if H < 1 or q.shape[-1] % H or q.shape[-1] == 0:
        raise ValueError(f"width {q.shape[-1]} is not divisible by {H} heads")
    d = q.shape[-1] // H
    if k is not None:
        _shaped(k, (*lead, Hk * d), "k")
        _same(q, k)
    for g, what in ((gamma_q, "gamma_q"), (gamma_k, "gamma_k")):
        if g is not None:
            _shaped(g, (d,), what)
    rot = 0
    if freqs is not None:
        rot = 2 * freqs.numel()
        if freqs.dim() != 1 or rot > d:
            raise ValueError(f"freqs must have shape (rot / 2,), rot <= {d}, not {tuple(freqs.shape)}")
        if pos is None:
            raise ValueError("a rotation needs pos")
        _integers(pos, lead, "pos")
    io = _io_of(q)
    dev = _target_device(q)
    qo, ko = out if out is not None else (None, None)
    with torch.cuda.device(dev):
        q, ldq = _rows(q, dev)
        k, ldk = _rows(k, dev)
        if rot:
            freqs, pos = _par(freqs, dev), _act(pos if pos.dtype is torch.int32 else pos.to(torch.int32), dev)
        else:
            freqs = pos = None
        gamma_q, gamma_k = _par(gamma_q, dev), _par(gamma_k, dev)
        qo = _out_like(qo, (*lead, H * d), q.dtype, dev)
        ko = None if k is None else _out_like(ko, (*lead, Hk * d), q.dtype, dev)
        _check(lr_head_norm_rope(_ptr(q), ldq, _ptr(k), ldk, _ptr(gamma_q), _ptr(gamma_k), _ptr(freqs), _ptr(pos),
                                 _ptr(qo), _ptr(ko), q.numel() // (H * d), H, Hk, d, rot, n, float(eps), p, io,
                                 _stream_of(q)), "lr_head_norm_rope")
    return qo, ko


def _step_state(state, shape, dev, state_out):
    """(state before the step or None, state buffer the step writes)."""
    h_in = None if state is None else _dev(state.float(), dev)
    if state_out is None:
        state_out = torch.empty(shape, dtype=torch.float32, device=dev)
    elif (tuple(state_out.shape) != tuple(shape) or state_out.dtype != torch.float32
          or state_out.device != dev or not state_out.is_contiguous()):
        raise ValueError(f"state_out must be a contiguous fp32 GPU tensor of shape {tuple(shape)}")
    return h_in, state_out


def selective_scan_step(x, dt, Bm, Cm, A_log, z=None, Dskip=None, h=None,
                        dt_softplus: bool = True, h_out=None):
    """One decode step of the selective SSM.  x, dt, z: (B, D); Bm, Cm: (B, 16),
    one dtype on the GPU; A_log: (D, 16); Dskip: (D,); h: (B, D, 16) fp32 or
    None (zero).  Returns (y (B, D), h_new (B, D, 16) fp32); ``h_out`` gives
    the buffer h_new is written to (it may be ``h`` itself)."""
    dev = _target_device(x)
    x, dt, z, Bm, Cm = (_dev(t, dev) for t in (x, dt, z, Bm, Cm))
    A_log, Dskip = (_dev(None if t is None else t.float(), dev) for t in (A_log, Dskip))
    _same(x, dt, z, Bm, Cm)
    B, D = x.shape
    N = Bm.shape[-1]
    h_in, h_new = _step_state(h, (B, D, N), dev, h_out)
    y = torch.empty_like(x)
    stream = torch.cuda.current_stream(dev).cuda_stream
    _check(lr_selective_scan_step(_ptr(x), _ptr(dt), _ptr(z), _ptr(Bm), _ptr(Cm), _ptr(A_log),
                                  _ptr(Dskip), _ptr(h_in), _ptr(h_new), _ptr(y), B, D, N,
                                  _io_of(x), int(bool(dt_softplus)), stream),
           "lr_selective_scan_step")
    return y, h_new


def rglru_scan_step(x, r, i, a_log, c: float = 8.0, h=None, h_out=None):
    """One decode step of the RG-LRU.  x, r, i: (B, D) on the GPU; a_log: (D,);
    h: (B, D) fp32 or None.  Returns (y (B, D), h_new (B, D) fp32)."""
    dev = _target_device(x)
    x, r, i = (_dev(t, dev) for t in (x, r, i))
    a_log = _dev(a_log.float(), dev)
    _same(x, r, i)
    B, D = x.shape
    h_in, h_new = _step_state(h, (B, D), dev, h_out)
    y = torch.empty_like(x)
    stream = torch.cuda.current_stream(dev).cuda_stream
    _check(lr_rglru_scan_step(_ptr(x), _ptr(r), _ptr(i), _ptr(a_log), float(c), _ptr(h_in),
                              _ptr(h_new), _ptr(y), B, D, _io_of(x), stream), "lr_rglru_scan_step")
    return y, h_new


def minmax_scan_step(r, s, x=None, x_out=None):
    """One decode step of the MinMax recurrence.  r, s: (B, D) on the GPU;
    x: (B, D) fp32 or None (zero).  Returns (y (B, D), x_new (B, D) fp32)."""
    dev = _target_device(r)
    r, s = (_dev(t, dev) for t in (r, s))
    _same(r, s)
    B, D = r.shape
    x_in, x_new = _step_state(x, (B, D), dev, x_out)
    y = torch.empty_like(r)
    stream = torch.cuda.current_stream(dev).cuda_stream
    _check(lr_minmax_scan_step(_ptr(r), _ptr(s), _ptr(x_in), _ptr(x_new), _ptr(y), B, D, _io_of(r),
                               stream), "lr_minmax_scan_step")
    return y, x_new


def hgrn2_step(q, k, v, g, H: int, S=None, S_out=None):
    """One decode step of HGRN2.  q, k: (B, H*dk); v, g: (B, H*dv) on the GPU;
    S: (B, H, dv, dk) fp32 or None.  Returns (o (B, H*dv), S_new)."""
    if q.shape[-1] % H or v.shape[-1] % H:
        raise ValueError(f"hidden size {q.shape[-1]} is not divisible by {H} heads")
    dev = _target_device(q)
    q, k, v, g = (_dev(t, dev) for t in (q, k, v, g))
    _same(q, k, v, g)
    B = q.shape[0]
    dk, dv = q.shape[-1] // H, v.shape[-1] // H
    S_in, S_new = _step_state(S, (B, H, dv, dk), dev, S_out)
    o = torch.empty(B, H * dv, dtype=q.dtype, device=dev)
    stream = torch.cuda.current_stream(dev).cuda_stream
    _check(lr_hgrn2_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(S_in), _ptr(S_new), _ptr(o),
                         B, H, dk, dv, _io_of(q), stream), "lr_hgrn2_step")
    return o, S_new


def decay_attn_step(q, k, v, H: int, Hk: Optional[int] = None, a_log=None, g=None, S=None, S_out=None,
                    scale: float = 1.0):
    """One token of ``decay_attn``.  q, k: (B, Hk*dk); v: (B, H*dv); g: (B, H)
    or None, one dtype on the GPU; a_log: (H,) fp32 or None; S: (B, H, dv, dk)
    fp32 or None (zero).  Returns (o (B, H*dv), S_new); ``S_out`` gives the
    buffer S_new is written to (it may be ``S`` itself)."""
    r = _lrtorch.decay_attn_step(q, k, v, H, Hk, a_log, g, S, S_out, scale)
    if type(r) is tuple:
        return r
    if r is not None:
        _check(r, "lr_decay_attn_step")
    (B, _), Hk, dk, dv, io = _heads_of(q, k, v, g, H, Hk, 2)
    shape = (B, H, dv, dk)
    if a_log is not None:
        _shaped(a_log, (H,), "a_log")
    if S is not None:
        _shaped(S, shape, "S")
    dev = _target_device(q)
    q, k, v, g = _act(q, dev), _act(k, dev), _act(v, dev), _act(g, dev)
    a_log, S = _par(a_log, dev), _par(S, dev)
    if S_out is None:
        S_out = torch.empty(shape, dtype=torch.float32, device=dev)
    elif S_out.shape != shape or S_out.dtype is not torch.float32 or S_out.device != dev or not S_out.is_contiguous():
        raise ValueError(f"S_out must be a contiguous fp32 GPU tensor of shape {shape}")
    o = torch.empty((B, H * dv), dtype=q.dtype, device=dev)
    rc = _lib.lr_decay_attn_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(a_log), _ptr(g), scale, _ptr(S),
                                 S_out.data_ptr(), o.data_ptr(), B, H, Hk, dk, dv, io, _stream_of(q))
    if rc != LR_OK:
        _check(rc, "lr_decay_attn_step")
    return o, S_out


def status(workspace=None, stream=None) -> int:
    """Device-side status code of the latest call that used ``workspace`` (a
    tensor; default: the workspace of this thread's latest call through the
    torch helpers); synchronises the stream (default: current) and resets
    the status to LR_OK."""
    ws = workspace if workspace is not None else last_workspace()
    if ws is None:
        return LR_OK
    s = (stream if stream is not None else torch.cuda.current_stream(ws.device)).cuda_stream
    return lr_check_status(ws.data_ptr(), s)


def check_status(workspace=None, stream=None) -> None:
    """As :func:`status`, raising :class:`LrError` on a non-zero code."""
    _check(status(workspace, stream), "device status")
