"""The torch helpers of the decayed attention, its step and the group norm as a
program calls them: views at any offset, calls that follow one another with nothing
between, an error that an earlier call left unread, and other Python threads."""
import ctypes
import threading
import time

import pytest
import torch

import oracle
from conftest import rel_err
from selective_state_space_chunked_gb300 import workloads as wl
from test_decay_attn_gpu import TOL, TOL_S, cuda, lr  # noqa: F401

pytestmark = pytest.mark.gpu


def step_args(p, t):
    return p["q"][:, t], p["k"][:, t], p["v"][:, t]


# ------------------------------------------------------------------ views
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_steps_on_views_of_one_row(lr, io):  # noqa: F811
    """[:, t] of one row is contiguous and starts anywhere."""
    L, H, dk, dv = 9, 6, 20, 12
    p = wl.decay_attn_inputs(1, L, H, dk, dv, seed=3, io=io, Hk=3, with_S0=True)
    a_log = torch.stack([p["a_log"]] * 3)
    d = cuda(p)
    S, outs = d["S0"].clone(), []
    for t in range(L):
        o, _ = lr.decay_attn_step(*step_args(d, t), H, Hk=3, a_log=a_log.cuda()[1], g=d["g"][:, t], S=S, S_out=S)
        outs.append(o[:, None])
    orf, Srf = oracle.decay_attn(p["q"], p["k"], p["v"], H, Hk=3, a_log=p["a_log"], g=p["g"], S0=p["S0"])
    assert rel_err(torch.cat(outs, 1).float().cpu(), orf) <= TOL[io] and rel_err(S.cpu(), Srf) <= TOL_S


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("host", [False, True])
def test_prompts_on_views(lr, io, host):  # noqa: F811
    L, H, d = 60, 3, 33
    p = wl.decay_attn_inputs(3, L, H, d, d, seed=4, io=io, with_S0=True)
    lens = torch.tensor([7, 60, 31], dtype=torch.int32)
    orf, Srf = oracle.decay_attn(p["q"], p["k"], p["v"], H, a_log=p["a_log"], g=p["g"], S0=p["S0"],
                                 lens=None if host else lens)
    q, k, v, g, S0 = (p[n] if host else p[n].cuda() for n in ("q", "k", "v", "g", "S0"))
    a_log = torch.stack([p["a_log"]] * 3)[1] if host else torch.stack([p["a_log"]] * 3).cuda()[1]
    if host:   # rows, steps of a row: contiguous from any offset
        o, S = lr.decay_attn(q[1:2, 1:], k[1:2, 1:], v[1:2, 1:], H, a_log=a_log, g=g[1:2, 1:], S0=S0[1:2])
        orf, Srf = oracle.decay_attn(p["q"][1:2, 1:], p["k"][1:2, 1:], p["v"][1:2, 1:], H, a_log=p["a_log"],
                                     g=p["g"][1:2, 1:], S0=p["S0"][1:2])
    else:
        o, S = lr.decay_attn(q[1:], k[1:], v[1:], H, a_log=a_log, g=g[1:], S0=S0[1:], lens=lens.cuda()[1:])
        orf, Srf = orf[1:], Srf[1:]
    assert rel_err(o.float().cpu(), orf) <= TOL[io] and rel_err(S.cpu(), Srf) <= TOL_S


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_group_norm_on_views(lr, io):  # noqa: F811
    gen = torch.Generator().manual_seed(2)
    x, z = (torch.randn(5, 33, generator=gen).to(torch.float32 if io == "f32" else torch.bfloat16) for _ in range(2))
    gamma = torch.randn(3, 33, generator=gen)
    y = lr.group_norm_act(x.cuda()[1:], 3, gamma=gamma.cuda()[1], z=z.cuda()[1:])
    # fp32: see test_group_norm_gpu; bf16: the store's rounding
    assert rel_err(y.float().cpu(), oracle.group_norm_act(x[1:], 3, gamma[1], None, z[1:])) <= {"f32": 5e-6,
                                                                                              "bf16": 4e-3}[io]
    with pytest.raises(lr.LrError):
        lr.group_norm_act(x.cuda(), 3, out=torch.empty(6, 33, dtype=x.dtype, device="cuda")[1:])
# ------------------------------------------- calls with nothing between them
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,dk,dv", [(1, 4, 64, 64), (16, 16, 128, 128), (300, 4, 32, 32), (7, 5, 33, 10)])
def test_calls_follow_one_another(lr, io, B, H, dk, dv):  # noqa: F811
    """prompt -> step -> step in place -> norm onto v -> step that reads it: each
    starts while the one before it drains, and reads what that one wrote."""
    n = 5
    p = wl.decay_attn_inputs(B, n, H, dk, dv, seed=B, io=io)
    d = cuda(p)
    qs, ks, gs = ([d[x][:, t].contiguous() for t in range(n)] for x in ("q", "k", "g"))
    vs = [d["v"][:, t].contiguous() for t in range(n)]
    prompt = [d[x][:, :1].contiguous() for x in ("q", "k", "v", "g")]
    a = d["a_log"]
    torch.cuda.synchronize()
    o, S = lr.decay_attn(*prompt[:3], H, a_log=a, g=prompt[3])
    outs = [o[:, 0]]
    for t in range(1, n):
        o, _ = lr.decay_attn_step(qs[t], ks[t], vs[t], H, a_log=a, g=gs[t], S=S, S_out=S)
        outs.append(o)
        if t + 1 < n:
            lr.group_norm_act(o, H, out=vs[t + 1])
    torch.cuda.synchronize()
    v = p["v"].clone()
    Sr, ref = None, []
    for t in range(n):   # the next v from the kernel's own output: no error is carried over
        orf, Sr = oracle.decay_attn(p["q"][:, t:t + 1], p["k"][:, t:t + 1], v[:, t:t + 1], H, a_log=p["a_log"],
                                    g=p["g"][:, t:t + 1], S0=Sr)
        assert rel_err(outs[t].float().cpu(), orf[:, 0]) <= TOL[io], t
        if 1 <= t < n - 1:
            want = oracle.group_norm_act(outs[t].float().cpu(), H)
            assert rel_err(vs[t + 1].float().cpu(), want) <= {"f32": 5e-6, "bf16": 4e-3}[io]
            v[:, t + 1] = vs[t + 1].cpu()
    assert rel_err(S.cpu(), Sr) <= TOL_S


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


# ---------------------------------------------------------------- threads
def test_other_threads_run_while_a_launch_waits(lr):  # noqa: F811
    """A launch onto a full queue waits for the GPU; Python's other threads do not.
    The queue is held for 1.5 s by a host function that needs no interpreter."""
    p = cuda(wl.decay_attn_inputs(1, 1, 2, 32, 32, 5, io="f32", with_S0=True))
    args, S = tuple(t.contiguous() for t in step_args(p, 0)), p["S0"]
    rt, libc = ctypes.CDLL("libcudart.so.13"), ctypes.CDLL(None)
    s = torch.cuda.Stream()
    stop, gaps = threading.Event(), [0.0]

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.002)
            now = time.perf_counter()
            gaps[0] = max(gaps[0], now - last)
            last = now

    with torch.cuda.stream(s):
        lr.decay_attn_step(*args, 2, S=S, S_out=S)
        s.synchronize()
        th = threading.Thread(target=tick)
        th.start()
        try:
            fn = ctypes.cast(libc.usleep, ctypes.c_void_p)
            assert rt.cudaLaunchHostFunc(ctypes.c_void_p(s.cuda_stream), fn, ctypes.c_void_p(1500000)) == 0
            t0 = time.perf_counter()
            for _ in range(4000):
                lr.decay_attn_step(*args, 2, S=S, S_out=S)
            waited = time.perf_counter() - t0
        finally:
            stop.set()
            th.join()
        s.synchronize()
    if waited < 1.0:
        pytest.skip("the queue took every launch")
    assert gaps[0] < 0.5
