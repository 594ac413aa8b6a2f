"""The torch helpers of the decayed attention, its step and the group norm as a
program calls them: errors."""
import ctypes

import pytest
import torch

from selective_state_space_chunked_gb300 import workloads as wl
from test_decay_attn_gpu import cuda, lr  # noqa: F401

pytestmark = pytest.mark.gpu


def step_args(p, t):
    return p["q"][:, t], p["k"][:, t], p["v"][:, t]


# ----------------------------------------------------------------- errors
@pytest.fixture
def unread_error():
    """Leaves an error in the calling thread's runtime state, as a failed call
    whose status nobody read does; cleared afterwards."""
    rt = ctypes.CDLL("libcudart.so.13")
    dev = torch.cuda.current_device()

    def leave():
        assert rt.cudaSetDevice(12345) != 0 and rt.cudaPeekAtLastError() != 0
        assert torch.cuda.current_device() == dev
    yield leave, rt.cudaGetLastError
    rt.cudaGetLastError()


def test_an_older_unread_error_repeats_no_call(lr, unread_error):  # noqa: F811
    leave, clear = unread_error
    p = cuda(wl.decay_attn_inputs(3, 1, 4, 32, 16, 5, io="f32", with_S0=True))
    args = tuple(t.contiguous() for t in step_args(p, 0))
    kw = dict(a_log=p["a_log"], g=p["g"][:, 0].contiguous())
    o, S1 = lr.decay_attn_step(*args, 4, S=p["S0"], **kw)
    S = p["S0"].clone()
    x = torch.randn(6, 64, device="cuda")
    y, xi = lr.group_norm_act(x, 4), x.clone()
    torch.cuda.synchronize()
    leave()
    lr.decay_attn_step(*args, 4, S=S, S_out=S, **kw)
    clear()
    leave()
    lr.group_norm_act(xi, 4, out=xi)
    clear()
    assert torch.equal(S, S1)    # one token, not two
    assert torch.equal(xi, y)


def test_a_failed_launch_is_raised_not_repeated(lr, monkeypatch):  # noqa: F811
    p = cuda(wl.decay_attn_inputs(2, 4, 2, 32, 32, 5, io="f32", with_S0=True))
    S = p["S0"].clone()
    for name in ("decay_attn", "decay_attn_step", "group_norm_act"):
        monkeypatch.setattr(lr._lrtorch, name, lambda *args: lr.LR_ERR_CUDA)
    with pytest.raises(lr.LrError):
        lr.decay_attn(p["q"], p["k"], p["v"], 2)
    with pytest.raises(lr.LrError):
        lr.decay_attn_step(*step_args(p, 0), 2, S=S, S_out=S)
    with pytest.raises(lr.LrError):
        lr.group_norm_act(S, 2, out=S)
    assert torch.equal(S, p["S0"])
