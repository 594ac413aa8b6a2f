"""Linear attention with a decay for each head (prompt and single-token forms)
against the float64 oracle, which runs the recurrence a step at a time.

Metric max|gpu - ref| / max|ref| on the outputs and on the state separately.
fp32 outputs and every state: sums of a few thousand products, each rounded to
2^-24, stay within 2e-5.  bf16 outputs: the store rounds to 2^-9, and the
decayed scores and the readout's copy of the state may be rounded to 2^-9 too:
1e-2, as for the other scans.
"""
import numpy as np
import pytest
import torch

import oracle
from conftest import rel_err
from selective_state_space_chunked_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
TOL = {"f32": 2e-5, "bf16": 1e-2}
TOL_S = 2e-5


@pytest.fixture(scope="module")
def lr():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_chunked_gb300 import build
    build.build()
    from selective_state_space_chunked_gb300 import binding
    return binding


def cuda(p):
    return {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in p.items()}


def check(lr, p, io, lens=None, scale=1.0, **kw):
    """Runs the call on p and compares outputs and state with the oracle."""
    d = cuda(p)
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    o, S = lr.decay_attn(d["q"], d["k"], d["v"], p["H"], Hk=p["Hk"], a_log=d["a_log"], g=d["g"], S0=d["S0"],
                         lens=None if n is None else n.cuda(), scale=scale, **kw)
    assert lr.status() == lr.LR_OK
    orf, Srf = oracle.decay_attn(p["q"], p["k"], p["v"], p["H"], Hk=p["Hk"], a_log=p["a_log"], g=p["g"],
                                 S0=p["S0"], lens=n, scale=scale)
    assert rel_err(o.float().cpu(), orf) <= TOL[io]
    assert rel_err(S.cpu(), Srf) <= TOL_S
    return o, S


# lengths around every tile and segment boundary: one step, a partial, a full
# and a just begun chunk of 16, 64 and 128 steps, and several of them
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 640, 1111])
def test_lengths(lr, io, L):
    check(lr, wl.decay_attn_inputs(2, L, 2, 128, 128, seed=L, io=io, with_S0=L % 2 == 0), io, scale=0.5)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("H,Hk,dk,dv", [
    (1, 1, 64, 64), (3, 3, 32, 64), (2, 2, 96, 192), (4, 2, 64, 128), (6, 1, 128, 64), (2, 2, 128, 256),
    (2, 2, 192, 64), (4, 4, 256, 128), (2, 1, 48, 72), (1, 1, 8, 8), (2, 2, 16, 40), (2, 2, 80, 24),
    (1, 1, 33, 17), (2, 1, 50, 100), (1, 1, 7, 3), (1, 1, 1, 1), (1, 1, 300, 20), (1, 1, 512, 16),
    (2, 2, 120, 136)])
def test_head_layouts(lr, io, H, Hk, dk, dv):
    check(lr, wl.decay_attn_inputs(2, 150, H, dk, dv, seed=dk + dv, io=io, Hk=Hk, with_S0=True), io)
    check(lr, wl.decay_attn_inputs(1, 5, H, dk, dv, seed=dk + dv + 1, io=io, Hk=Hk), io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("decay", ["none", "head", "token", "both"])
@pytest.mark.parametrize("with_S0", [True, False])
def test_decay_kinds(lr, io, decay, with_S0):
    check(lr, wl.decay_attn_inputs(2, 700, 4, 64, 64, seed=9, io=io, decay=decay, with_S0=with_S0), io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 200])
def test_ragged_rows(lr, io, d):
    """Row lengths of zero, one, a chunk's end and beyond the tensor; what
    stands past a row's length (NaN and infinities) does not reach it."""
    L = 389
    lens = [0, 1, 128, 129, 300, L, L + 50, -3]
    p = wl.decay_attn_inputs(len(lens), L, 2, d, 64, seed=3, io=io, with_S0=True)
    want = {n: p[n].clone() for n in ("q", "k", "v", "g")}
    for b, n in enumerate(lens):
        n = min(max(n, 0), L)
        for name, bad in (("q", float("nan")), ("k", float("inf")), ("v", float("nan")), ("g", float("nan"))):
            p[name][b, n:] = bad
            want[name][b, n:] = 0
    d_ = cuda(p)
    o, S = lr.decay_attn(d_["q"], d_["k"], d_["v"], 2, a_log=d_["a_log"], g=d_["g"], S0=d_["S0"],
                         lens=torch.tensor(lens).cuda())
    assert lr.status() == lr.LR_OK
    orf, Srf = oracle.decay_attn(want["q"], want["k"], want["v"], 2, a_log=p["a_log"], g=want["g"], S0=p["S0"],
                                 lens=np.array(lens))
    assert rel_err(o.float().cpu(), orf) <= TOL[io]
    assert rel_err(S.cpu(), Srf) <= TOL_S
    for b, n in enumerate(lens):
        assert torch.all(o[b, max(n, 0):] == 0)
    assert torch.equal(S[0].cpu(), p["S0"][0]) and torch.equal(S[-1].cpu(), p["S0"][-1])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 160])
def test_resets_and_steep_decays(lr, io, d):
    """Decays of 0 (log decay -inf and the type's lowest value), steps that
    decay by 2^-30 to 2^-140, and none at all, in one sequence."""
    L = 600
    p = wl.decay_attn_inputs(2, L, 3, d, 64, seed=17, io=io, with_S0=True)
    g = p["g"].float()
    gen = torch.Generator().manual_seed(1)
    at = torch.randperm(L, generator=gen)
    g[:, at[:8], 0] = -float("inf")
    g[:, at[8:16], 0] = torch.finfo(torch.float32).min if io == "f32" else torch.finfo(torch.bfloat16).min
    g[:, at[:200], 1] = -100.0 * torch.rand(2, 200, generator=gen) - 20.0
    g[:, 100:300, 2] = -3.0
    g[:, 300:500, 2] = 0.0
    g[0, 0, 0] = -float("inf")
    p["g"] = g.to(p["g"].dtype)
    check(lr, p, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_long_memory_does_not_drift(lr, io):
    """Decays of 1 - 2^-12 remember thousands of steps: a factor rounded the
    same way at every chunk would show in the state."""
    check(lr, wl.decay_attn_inputs(1, 9000, 2, 64, 64, seed=21, io=io, decay="head", with_S0=True), io)
    p = wl.decay_attn_inputs(1, 9000, 1, 64, 64, seed=22, io=io, decay="head")
    p["a_log"] = torch.full((1,), -2.0 ** -13)
    check(lr, p, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("cut", [1, 64, 100, 383])
def test_resume_from_the_final_state(lr, io, cut):
    p = wl.decay_attn_inputs(2, 384, 2, 128, 64, seed=5, io=io)
    d = cuda(p)
    parts, S = [], None
    for sl in (slice(0, cut), slice(cut, 384)):
        o, S = lr.decay_attn(d["q"][:, sl], d["k"][:, sl], d["v"][:, sl], 2, a_log=d["a_log"], g=d["g"][:, sl], S0=S)
        parts.append(o)
    orf, Srf = oracle.decay_attn(p["q"], p["k"], p["v"], 2, a_log=p["a_log"], g=p["g"])
    assert rel_err(torch.cat(parts, 1).float().cpu(), orf) <= TOL[io]
    assert rel_err(S.cpu(), Srf) <= TOL_S


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,L,d", [(1, 1, 8192, 64), (1, 2, 5000, 128), (2, 3, 3001, 96)])
def test_few_heads_long_sequences_run_in_segments(lr, io, B, H, L, d):
    p = wl.decay_attn_inputs(B, L, H, d, d, seed=8, io=io, with_S0=True)
    ws = lr.lr_decay_attn_workspace_size(B, L, H, H, d, d, lr.LR_BF16 if io == "bf16" else lr.LR_F32)
    assert ws > 256
    check(lr, p, io)
    check(lr, p, io, lens=[L // 3] * B)


def test_large_values_keep_their_scale(lr):
    """v k products of 2^40 and 2^-40 go through the scaled state alike."""
    for e in (20.0, -20.0):
        p = wl.decay_attn_inputs(1, 300, 2, 64, 64, seed=4, io="f32")
        p["k"], p["v"] = p["k"] * 2.0 ** e, p["v"] * 2.0 ** e
        check(lr, p, "f32")


def test_non_contiguous_inputs_and_out(lr):
    B, L, H, d = 2, 200, 2, 64
    p = wl.decay_attn_inputs(B, L, H, d, d, seed=6, io="bf16")
    packed = torch.cat([p["q"], p["k"], p["v"]], -1).cuda()     # views of one projection
    q, k, v = packed.split(H * d, -1)
    assert not q.is_contiguous()
    g = p["g"].transpose(1, 2).contiguous().cuda().transpose(1, 2)
    o = torch.empty(B, L, H * d, dtype=torch.bfloat16, device="cuda")
    S = torch.empty(B, H, d, d, device="cuda")
    res = lr.decay_attn(q, k, v, H, a_log=p["a_log"].cuda(), g=g, out=(o, S))
    assert res[0] is o and res[1] is S
    orf, Srf = oracle.decay_attn(p["q"], p["k"], p["v"], H, a_log=p["a_log"], g=p["g"])
    assert rel_err(o.float().cpu(), orf) <= TOL["bf16"] and rel_err(S.cpu(), Srf) <= TOL_S


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_another_stream_and_a_dirty_workspace(lr, io):
    p = wl.decay_attn_inputs(1, 3000, 2, 128, 128, seed=7, io=io)
    ws = torch.full((lr.lr_decay_attn_workspace_size(1, 3000, 2, 2, 128, 128, 1 if io == "bf16" else 0),), 255,
                    dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        first = check(lr, p, io, workspace=ws)
        again = check(lr, p, io, workspace=ws)
    s.synchronize()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])   # a fixed order of sums


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 33])
@pytest.mark.parametrize("value", [0.5, float("nan"), float("inf")])
def test_log_decays_out_of_range_are_reported(lr, io, d, value):
    p = cuda(wl.decay_attn_inputs(1, 200, 2, d, d, seed=2, io=io))
    p["g"][0, 150, 1] = value
    lr.decay_attn(p["q"], p["k"], p["v"], 2, a_log=p["a_log"], g=p["g"])
    assert lr.status() == lr.LR_ERR_RANGE
    p["g"][0, 150, 1] = -0.5
    lr.decay_attn(p["q"], p["k"], p["v"], 2, a_log=p["a_log"], g=p["g"])
    assert lr.status() == lr.LR_OK


def test_empty_problems(lr):
    z = torch.zeros(2, 0, 64, device="cuda")
    S0 = torch.randn(2, 1, 64, 64, device="cuda")
    o, S = lr.decay_attn(z, z, z, 1, S0=S0)
    assert o.shape == (2, 0, 64) and torch.equal(S, S0)
    assert lr.status() == lr.LR_OK
    o, S = lr.decay_attn(z, z, z, 1)
    assert torch.all(S == 0)
    e = torch.zeros(0, 5, 64, device="cuda")
    o, S = lr.decay_attn(e, e, e, 1)
    assert o.shape == (0, 5, 64) and S.shape == (0, 1, 64, 64)


def test_captured_in_a_graph(lr):
    p = wl.decay_attn_inputs(1, 2000, 2, 128, 128, seed=12, io="bf16")
    d = cuda(p)
    o = torch.empty(1, 2000, 256, dtype=torch.bfloat16, device="cuda")
    S = torch.empty(1, 2, 128, 128, device="cuda")
    ws = torch.empty(lr.lr_decay_attn_workspace_size(1, 2000, 2, 2, 128, 128, 1), dtype=torch.uint8, device="cuda")
    args = (d["q"], d["k"], d["v"], 2)
    kw = dict(a_log=d["a_log"], g=d["g"], workspace=ws, out=(o, S))
    lr.decay_attn(*args, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lr.decay_attn(*args, **kw)
    o.zero_(), S.zero_()
    graph.replay()
    torch.cuda.synchronize()
    orf, Srf = oracle.decay_attn(p["q"], p["k"], p["v"], 2, a_log=p["a_log"], g=p["g"])
    assert rel_err(o.float().cpu(), orf) <= TOL["bf16"] and rel_err(S.cpu(), Srf) <= TOL_S


# ------------------------------------------------------------ host buffers
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("queued", [False, True])
@pytest.mark.parametrize("decay", ["head", "token", "none"])
def test_host_buffers_in_chunks(lr, io, queued, decay):
    p = wl.decay_attn_inputs(2, 500, 4, 64, 32, seed=14, io=io, Hk=2, decay=decay, with_S0=True)
    prev = lr.lr_set_host_chunk_steps(192)
    try:
        o, S = lr.decay_attn(p["q"], p["k"], p["v"], 4, Hk=2, a_log=p["a_log"], g=p["g"], S0=p["S0"],
                             sync_host=not queued)
        if queued:
            lr.host_sync()
    finally:
        lr.lr_set_host_chunk_steps(prev)
    assert not o.is_cuda and not S.is_cuda
    orf, Srf = oracle.decay_attn(p["q"], p["k"], p["v"], 4, Hk=2, a_log=p["a_log"], g=p["g"], S0=p["S0"])
    assert rel_err(o.float(), orf) <= TOL[io] and rel_err(S, Srf) <= TOL_S


def test_host_tensors_with_lengths(lr):
    p = wl.decay_attn_inputs(2, 90, 2, 64, 64, seed=15, io="f32")
    o, S = lr.decay_attn(p["q"], p["k"], p["v"], 2, a_log=p["a_log"], g=p["g"], lens=torch.tensor([90, 31]))
    orf, Srf = oracle.decay_attn(p["q"], p["k"], p["v"], 2, a_log=p["a_log"], g=p["g"], lens=[90, 31])
    assert not o.is_cuda
    assert rel_err(o, orf) <= TOL["f32"] and rel_err(S, Srf) <= TOL_S


# ------------------------------------------------------------ one token
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,Hk,dk,dv", [
    (1, 16, 16, 128, 128), (64, 16, 16, 128, 128), (17, 24, 8, 64, 128), (3, 4, 4, 32, 64), (2, 2, 1, 96, 192),
    (5, 3, 3, 256, 64), (2, 2, 2, 33, 17), (1, 1, 1, 1, 1), (9, 2, 2, 20, 5), (300, 4, 2, 64, 64),
    (2, 1, 1, 600, 4), (40, 8, 8, 16, 200)])
@pytest.mark.parametrize("decay", ["both", "none"])
def test_step(lr, io, B, H, Hk, dk, dv, decay):
    p = wl.decay_attn_inputs(B, 1, H, dk, dv, seed=B + dk, io=io, Hk=Hk, decay=decay, with_S0=True)
    d = cuda(p)
    g = None if d["g"] is None else d["g"][:, 0]
    o, S = lr.decay_attn_step(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], H, Hk=Hk, a_log=d["a_log"], g=g,
                              S=d["S0"], scale=0.7)
    orf, Srf = oracle.decay_attn(p["q"], p["k"], p["v"], H, Hk=Hk, a_log=p["a_log"], g=p["g"], S0=p["S0"],
                                 scale=0.7)
    assert rel_err(o.float().cpu()[:, None], orf) <= TOL[io]
    assert rel_err(S.cpu(), Srf) <= TOL_S
    o0, S0 = lr.decay_attn_step(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], H, Hk=Hk, a_log=d["a_log"], g=g,
                                scale=0.7)
    orf, Srf = oracle.decay_attn(p["q"], p["k"], p["v"], H, Hk=Hk, a_log=p["a_log"], g=p["g"], scale=0.7)
    assert rel_err(o0.float().cpu()[:, None], orf) <= TOL[io]
    assert rel_err(S0.cpu(), Srf) <= TOL_S


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (50, 30)])
def test_steps_in_place_continue_a_prompt(lr, io, dk, dv):
    L, n, H = 140, 130, 2
    p = wl.decay_attn_inputs(2, L, H, dk, dv, seed=31, io=io)
    d = cuda(p)
    o, S = lr.decay_attn(d["q"][:, :n], d["k"][:, :n], d["v"][:, :n], H, a_log=d["a_log"], g=d["g"][:, :n])
    outs = [o]
    for t in range(n, L):
        o, S2 = lr.decay_attn_step(d["q"][:, t], d["k"][:, t], d["v"][:, t], H, a_log=d["a_log"], g=d["g"][:, t],
                                   S=S, S_out=S)
        assert S2 is S
        outs.append(o[:, None])
    orf, Srf = oracle.decay_attn(p["q"], p["k"], p["v"], H, a_log=p["a_log"], g=p["g"])
    assert rel_err(torch.cat(outs, 1).float().cpu(), orf) <= TOL[io]
    assert rel_err(S.cpu(), Srf) <= TOL_S


def test_step_reset_clears_the_state(lr):
    p = cuda(wl.decay_attn_inputs(2, 1, 2, 64, 64, seed=33, io="f32", with_S0=True))
    args = (p["q"][:, 0], p["k"][:, 0], p["v"][:, 0], 2)
    g = torch.full((2, 2), -float("inf"), device="cuda")
    a, b = lr.decay_attn_step(*args, g=g, S=p["S0"]), lr.decay_attn_step(*args)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_offsets_past_two_to_the_31(lr):
    """8192 value channels per step and 2 x 270,001 steps: 4.4e9 elements of v
    and o.  The last row's first and last heads against the oracle."""
    B, L, H, dk, dv = 2, 270001, 64, 32, 128
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k = (torch.randn(B, L, dk, generator=gen, device="cuda").bfloat16() / dk ** 0.5 for _ in range(2))
    v = torch.empty(B, L, H * dv, dtype=torch.bfloat16, device="cuda")
    for i in range(0, L, 30000):
        v[:, i:i + 30000] = torch.randn(B, min(30000, L - i), H * dv, generator=gen, device="cuda") / 11.0
    a_log = torch.linspace(-0.5, -0.02, H, device="cuda")
    o, S = lr.decay_attn(q, k, v, H, Hk=1, a_log=a_log)
    assert lr.status() == lr.LR_OK
    n = 3000   # decays of at most exp(-0.02 n): what came before is gone
    for h in (0, H - 1):
        c = slice(h * dv, (h + 1) * dv)
        orf, Srf = oracle.decay_attn(q[-1:, -n:].cpu(), k[-1:, -n:].cpu(), v[-1:, -n:, c].cpu(), 1,
                                     a_log=a_log[h:h + 1].cpu())
        assert rel_err(o[-1:, -n // 2:, c].float().cpu(), orf[:, -n // 2:]) <= TOL["bf16"]
        assert rel_err(S[-1:, h:h + 1].cpu(), Srf) <= TOL_S
