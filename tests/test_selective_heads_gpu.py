"""Selective scan with heads (prompt and single-token forms) against the float64 oracle.

Metric max|gpu - ref| / max|ref| on the outputs and on the state separately.  The
recurrence is the decayed attention's, whose bounds hold (see test_decay_attn_gpu): 2e-5
for fp32 outputs and every state; the step size adds 4 * 2^-24 of a log decay l to it, and
so l e^-l 4 * 2^-24 < 1e-7 to what is left of a state.  bf16 outputs: the store's half step of 2^-8, and the rounded scores (the skip
among them) and state copy, 2^-8 each of their own term: 1e-2.
"""
import numpy as np
import pytest
import torch

import oracle
from conftest import rel_err
from selective_state_space_chunked_gb300 import workloads as wl
from test_decay_attn_gpu import cuda, lr  # noqa: F401

pytestmark = pytest.mark.gpu
TOL = {"f32": 2e-5, "bf16": 1e-2}
TOL_S = 2e-5
NAMES = ("x", "dt", "Bm", "Cm")
OPT = ("z", "Dskip", "dt_bias", "S0")


def check(lr, p, io, lens=None, **kw):  # noqa: F811
    d = cuda(p)
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    y, S = lr.selective_heads(*(d[k] for k in NAMES), d["A_log"], p["H"], G=p["G"], lens=None if n is None else n.cuda(),
                              **{k: d[k] for k in OPT}, **kw)
    assert lr.status() == lr.LR_OK
    yr, Sr = oracle.selective_heads(*(p[k] for k in NAMES), p["A_log"], p["H"], G=p["G"], lens=lens,
                                    **{k: p[k] for k in OPT}, **{k: v for k, v in kw.items() if k == "dt_softplus"})
    assert rel_err(y.float().cpu(), yr) <= TOL[io]
    assert rel_err(S.cpu(), Sr) <= TOL_S
    return y, S


# lengths around every tile and segment boundary
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 47, 48, 63, 64, 65, 127, 128, 129, 255, 257, 640, 1111])
def test_lengths(lr, io, L):  # noqa: F811
    check(lr, wl.selective_heads_inputs(2, L, 4, 1, 64, 128, seed=L, io=io, z=L % 3 != 0, skip=L % 4 != 1,
                                        with_S0=L % 2 == 0), io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("H,G,P,N", [
    (1, 1, 64, 64), (3, 3, 64, 32), (2, 2, 192, 96), (4, 2, 128, 64), (6, 1, 64, 128), (2, 2, 256, 128), (2, 2, 64, 192),
    (4, 4, 128, 256), (2, 1, 72, 48), (1, 1, 8, 8), (2, 2, 40, 16), (2, 2, 24, 80), (1, 1, 17, 33), (2, 1, 100, 50),
    (1, 1, 3, 7), (1, 1, 1, 1), (1, 1, 20, 300), (1, 1, 16, 512), (2, 2, 136, 120), (8, 2, 32, 16)])
def test_head_layouts(lr, io, H, G, P, N):  # noqa: F811
    check(lr, wl.selective_heads_inputs(2, 150, H, G, P, N, seed=P + N, io=io, with_S0=True), io)
    check(lr, wl.selective_heads_inputs(1, 5, H, G, P, N, seed=P + N + 1, io=io, z=False), io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("N", [64, 160])
@pytest.mark.parametrize("z,skip,bias,S0", [(True, False, True, False), (False, True, False, True),
                                            (False, False, False, False), (True, True, False, True)])
def test_what_may_be_absent(lr, io, N, z, skip, bias, S0):  # noqa: F811
    p = wl.selective_heads_inputs(2, 300, 4, 2, 72, N, seed=9, io=io, z=z, skip=skip, with_S0=S0)
    if not bias:
        p["dt_bias"], p["dt"] = None, (p["dt"].float() - 4.0).to(p["dt"].dtype)
    check(lr, p, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("N", [64, 128, 200])
def test_ragged_rows(lr, io, N):  # noqa: F811
    """Row lengths of zero, one, a chunk's end and beyond the tensor; what stands past
    a row's length (NaN and infinities) does not reach it."""
    L = 389
    lens = [0, 1, 128, 129, 300, L, L + 50, -3]
    p = wl.selective_heads_inputs(len(lens), L, 2, 1, 64, N, seed=3, io=io, with_S0=True)
    for b, n in enumerate(lens):
        for name, bad in (("x", float("nan")), ("Bm", float("inf")), ("Cm", float("nan")), ("dt", float("nan")),
                          ("z", float("nan"))):
            p[name][b, min(max(n, 0), L):] = bad
    y, S = check(lr, p, io, lens=lens)
    for b, n in enumerate(lens):
        assert torch.all(y[b, max(n, 0):] == 0)
    assert torch.equal(S[0].cpu(), p["S0"][0]) and torch.equal(S[-1].cpu(), p["S0"][-1])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("N", [64, 128, 160])
def test_large_and_small_step_sizes(lr, io, N):  # noqa: F811
    """Steps of 0 (nothing enters or decays), resets, steep chunks and slow ones."""
    L = 600
    p = wl.selective_heads_inputs(2, L, 4, 2, 64, N, seed=17, io=io, with_S0=True)
    gen = torch.Generator().manual_seed(1)
    dt = p["dt"].float()
    at = torch.randperm(L, generator=gen)
    dt[:, at[:30]] = -float("inf")                       # delta = 0
    dt[:, at[30:40], 0] = 300.0
    dt[:, at[:200], 1] = 3.0 + 10.0 * torch.rand(2, 200, generator=gen)
    dt[:, 100:300, 2] = 6.0
    dt[:, 300:500, 2] = -20.0
    p["dt"] = dt.to(p["dt"].dtype)
    check(lr, p, io)


@pytest.mark.parametrize("io,B,L,H,G,P,N", [
    ("f32", 1, 90, 4, 1, 64, 128), ("f32", 1, 333, 2, 1, 24, 20), ("f32", 2, 700, 12, 3, 80, 96), ("f32", 4, 37, 16, 1, 128, 128),
    ("f32", 8, 101, 16, 4, 64, 128), ("f32", 5, 203, 9, 3, 70, 250), ("f32", 3, 411, 6, 1, 33, 61), ("f32", 32, 50, 16, 2, 64, 64),
    ("f32", 2, 150, 8, 2, 64, 32), ("bf16", 1, 40, 16, 2, 128, 128), ("bf16", 8, 47, 16, 1, 64, 128), ("bf16", 2, 300, 5, 5, 50, 60)])
@pytest.mark.parametrize("ragged", [False, True])
def test_rows_a_thread_and_segments(lr, io, B, L, H, G, P, N, ragged):  # noqa: F811
    """Few blocks and many, one segment and several, aligned rows and others; heads that
    hardly decay beside heads whose every chunk decays below 2^-32."""
    p = wl.selective_heads_inputs(B, L, H, G, P, N, seed=L + N, io=io, with_S0=True)
    dt = p["dt"].float()
    dt[..., 0] = 4.0
    if H > 2:
        dt[..., 1] = -12.0
        dt[:, L // 3:, 2] = 2.0
    p["dt"] = dt.to(p["dt"].dtype)
    lens = [(L * (b + 1) * 7) % (L + 1) for b in range(B)] if ragged else None
    check(lr, p, io, lens=lens)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_step_sizes_given_as_they_are(lr, io):  # noqa: F811
    p = wl.selective_heads_inputs(2, 200, 2, 1, 64, 64, seed=4, io=io)
    p["dt"] = torch.nn.functional.softplus(p["dt"].float() - 3.0).to(p["dt"].dtype)
    p["dt_bias"] = torch.tensor([0.0, 0.01])
    check(lr, p, io, dt_softplus=False)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("N", [64, 33, 192])
def test_step_sizes_out_of_range_are_reported(lr, io, N):  # noqa: F811
    p = wl.selective_heads_inputs(1, 200, 2, 1, 64, N, seed=2, io=io)
    good = p["dt"].clone()
    for value, soft, code in ((float("nan"), True, -7), (-0.5, False, -7), (0.5, False, 0), (-0.5, True, 0),
                              (float("nan"), False, -7)):
        p["dt"] = good.abs() if not soft else good.clone()
        p["dt"][0, 150, 1] = value
        if not soft:
            p["dt_bias"] = None
        d = cuda(p)
        lr.selective_heads(*(d[k] for k in NAMES), d["A_log"], 2, dt_softplus=soft, dt_bias=d["dt_bias"])
        assert lr.status() == code, (value, soft)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_long_memory_does_not_drift(lr, io):  # noqa: F811
    p = wl.selective_heads_inputs(1, 9000, 2, 1, 64, 64, seed=21, io=io, with_S0=True, rate=(0.002, 0.05))
    check(lr, p, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,L,P,N", [(1, 1, 8192, 64, 64), (1, 2, 5000, 128, 128), (2, 3, 3001, 96, 96),
                                       (1, 2, 4000, 64, 256)])
def test_few_heads_long_sequences_run_in_segments(lr, io, B, H, L, P, N):  # noqa: F811
    p = wl.selective_heads_inputs(B, L, H, 1, P, N, seed=8, io=io, with_S0=True, rate=(0.1, 4.0))
    assert lr.lr_selective_heads_workspace_size(B, L, H, 1, P, N, lr.LR_BF16 if io == "bf16" else lr.LR_F32) > 256
    check(lr, p, io)
    check(lr, p, io, lens=[L // 3] * B)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("cut", [1, 64, 100, 383])
def test_resume_from_the_final_state(lr, io, cut):  # noqa: F811
    p = wl.selective_heads_inputs(2, 384, 2, 1, 64, 128, seed=5, io=io)
    d = cuda(p)
    parts, S = [], None
    for sl in (slice(0, cut), slice(cut, 384)):
        y, S = lr.selective_heads(*(d[k][:, sl] for k in NAMES), d["A_log"], 2, z=d["z"][:, sl], Dskip=d["Dskip"],
                                  dt_bias=d["dt_bias"], S0=S)
        parts.append(y)
    yr, Sr = oracle.selective_heads(*(p[k] for k in NAMES), p["A_log"], 2, **{k: p[k] for k in OPT})
    assert rel_err(torch.cat(parts, 1).float().cpu(), yr) <= TOL[io] and rel_err(S.cpu(), Sr) <= TOL_S


# ------------------------------------------------------------ where rows stand
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("P,N,apart", [(64, 128, 0), (64, 64, 8), (32, 16, 3), (80, 96, 5), (10, 12, 0)])
@pytest.mark.parametrize("L", [30, 200])
def test_slices_of_wider_tensors(lr, io, P, N, apart, L):  # noqa: F811
    """x, B and C of one convolution's output, z and dt of one projection's: read where
    they stand, or copied where rows leave 16-byte boundaries."""
    H, G = 4, 2
    p = wl.selective_heads_inputs(3, L, H, G, P, N, seed=P, io=io, with_S0=True)
    d = cuda(p)
    pad = torch.full((3, L, apart), float("nan"), dtype=d["x"].dtype, device="cuda")
    xbc = torch.cat([d["x"], d["Bm"], d["Cm"], pad], -1)
    zdt = torch.cat([d["z"], pad, d["dt"]], -1)
    x, Bm, Cm = xbc[..., :H * P], xbc[..., H * P:H * P + G * N], xbc[..., H * P + G * N:H * P + 2 * G * N]
    z, dt = zdt[..., :H * P], zdt[..., H * P + apart:]
    y, S = lr.selective_heads(x, dt, Bm, Cm, d["A_log"], H, G=G, z=z, Dskip=d["Dskip"], dt_bias=d["dt_bias"], S0=d["S0"])
    lr.check_status()
    yr, Sr = oracle.selective_heads(*(p[k] for k in NAMES), p["A_log"], H, G=G, **{k: p[k] for k in OPT})
    assert rel_err(y.float().cpu(), yr) <= TOL[io] and rel_err(S.cpu(), Sr) <= TOL_S
    S1 = d["S0"].clone()
    y1, _ = lr.selective_heads_step(x[:, 0], dt[:, 0], Bm[:, 0], Cm[:, 0], d["A_log"], H, G=G, z=z[:, 0],
                                    Dskip=d["Dskip"], dt_bias=d["dt_bias"], S=S1, S_out=S1)
    yr, Sr = oracle.selective_heads(*(p[k][:, :1] for k in NAMES), p["A_log"], H, G=G, z=p["z"][:, :1],
                                    Dskip=p["Dskip"], dt_bias=p["dt_bias"], S0=p["S0"])
    assert rel_err(y1.float().cpu()[:, None], yr) <= TOL[io] and rel_err(S1.cpu(), Sr) <= TOL_S


def test_another_stream_a_dirty_workspace_and_a_graph(lr):  # noqa: F811
    p = wl.selective_heads_inputs(1, 3000, 2, 1, 128, 128, seed=7, io="bf16")
    d = cuda(p)
    ws = torch.full((lr.lr_selective_heads_workspace_size(1, 3000, 2, 1, 128, 128, 1),), 255, dtype=torch.uint8,
                    device="cuda")
    y, S = torch.empty_like(d["x"]), torch.empty(1, 2, 128, 128, device="cuda")
    call = lambda: lr.selective_heads(*(d[k] for k in NAMES), d["A_log"], 2, workspace=ws, out=(y, S),  # noqa: E731
                                      **{k: d[k] for k in OPT})
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
        side.synchronize()
        first = y.clone(), S.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    for _ in range(2):
        y.zero_(), S.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, first[0]) and torch.equal(S, first[1])   # a fixed order of sums
    yr, Sr = oracle.selective_heads(*(p[k] for k in NAMES), p["A_log"], 2, **{k: p[k] for k in OPT})
    assert rel_err(y.float().cpu(), yr) <= TOL["bf16"] and rel_err(S.cpu(), Sr) <= TOL_S


def test_empty_problems(lr):  # noqa: F811
    z = torch.zeros(2, 0, 64, device="cuda")
    S0, a = torch.randn(2, 1, 64, 64, device="cuda"), torch.zeros(1, device="cuda")
    y, S = lr.selective_heads(z, z[..., :1], z, z, a, 1, S0=S0)
    assert y.shape == (2, 0, 64) and torch.equal(S, S0) and lr.status() == lr.LR_OK
    y, S = lr.selective_heads(z, z[..., :1], z, z, a, 1)
    assert torch.all(S == 0)
    e = torch.zeros(0, 5, 64, device="cuda")
    y, S = lr.selective_heads(e, e[..., :1], e, e, a, 1)
    assert y.shape == (0, 5, 64) and S.shape == (0, 1, 64, 64)


# ------------------------------------------------------- infinities and NaN
def same_values(lr, p, io, lens=None):  # noqa: F811
    d = cuda(p)
    y, S = lr.selective_heads(*(d[k] for k in NAMES), d["A_log"], p["H"], G=p["G"],
                              lens=None if lens is None else torch.tensor(lens).cuda(), **{k: d[k] for k in OPT})
    assert lr.status() == lr.LR_OK
    with np.errstate(invalid="ignore"):
        yr, Sr = oracle.selective_heads(*(p[k] for k in NAMES), p["A_log"], p["H"], G=p["G"], lens=lens,
                                        **{k: p[k] for k in OPT})
    for got, want, tol in ((y.double().cpu().numpy(), yr, TOL[io]), (S.double().cpu().numpy(), Sr, TOL_S)):
        finite = np.isfinite(want)
        assert np.array_equal(np.isfinite(got), finite)
        if finite.any():
            assert np.max(np.abs(got[finite] - want[finite])) <= tol * np.max(np.abs(want[finite]))
    return y, S


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("N", [64, 128, 200])
@pytest.mark.parametrize("which", ["x", "Bm", "Cm", "z"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_bad_value_reaches_no_earlier_step(lr, io, N, which, value):  # noqa: F811
    p = wl.selective_heads_inputs(2, 300, 2, 1, 64, N, seed=5, io=io, with_S0=True, rate=(0.1, 1.0))
    p[which][0, 200, 3] = value
    y, _ = same_values(lr, p, io)
    assert torch.isfinite(y[0, :200]).all() and torch.isfinite(y[1]).all()
    assert not torch.isfinite(y[0, 200, 3])
    if which == "z":
        assert int((~torch.isfinite(y)).sum()) == 1


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("N", [64, 192])
def test_bad_values_in_segments(lr, io, N):  # noqa: F811
    p = wl.selective_heads_inputs(1, 5000, 2, 1, 64, N, seed=6, io=io, with_S0=True, rate=(0.05, 0.1))
    p["x"][0, 777, 3], p["x"][0, 4999, 70], p["Bm"][0, 2500, N - 1] = float("inf"), float("nan"), -float("inf")
    p["S0"][0, 1, 9, 2] = float("nan")
    same_values(lr, p, io)
    same_values(lr, p, io, lens=[4321])


# ------------------------------------------------------------ one token
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,G,P,N", [
    (1, 16, 1, 128, 128), (64, 16, 1, 128, 128), (17, 24, 8, 128, 64), (3, 4, 4, 64, 32), (2, 2, 1, 192, 96),
    (5, 3, 3, 64, 256), (2, 2, 2, 17, 33), (1, 1, 1, 1, 1), (9, 2, 2, 5, 20), (300, 4, 2, 64, 64), (2, 1, 1, 4, 600),
    (40, 8, 8, 200, 16)])
@pytest.mark.parametrize("full", [True, False])
def test_step(lr, io, B, H, G, P, N, full):  # noqa: F811
    p = wl.selective_heads_inputs(B, 1, H, G, P, N, seed=B + N, io=io, z=full, skip=full, with_S0=full)
    d = cuda(p)
    y, S = lr.selective_heads_step(*(d[k][:, 0] for k in NAMES), d["A_log"], H, G=G, z=d["z"][:, 0] if full else None,
                                   Dskip=d["Dskip"], dt_bias=d["dt_bias"], S=d["S0"])
    yr, Sr = oracle.selective_heads(*(p[k] for k in NAMES), p["A_log"], H, G=G, **{k: p[k] for k in OPT})
    assert rel_err(y.float().cpu()[:, None], yr) <= TOL[io] and rel_err(S.cpu(), Sr) <= TOL_S


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("P,N", [(128, 128), (64, 128), (30, 50)])
def test_steps_in_place_continue_a_prompt(lr, io, P, N):  # noqa: F811
    L, n, H = 140, 130, 2
    p = wl.selective_heads_inputs(2, L, H, 1, P, N, seed=31, io=io)
    d = cuda(p)
    kw = dict(Dskip=d["Dskip"], dt_bias=d["dt_bias"])
    y, S = lr.selective_heads(*(d[k][:, :n] for k in NAMES), d["A_log"], H, z=d["z"][:, :n], **kw)
    outs = [y]
    for t in range(n, L):
        y, S2 = lr.selective_heads_step(*(d[k][:, t] for k in NAMES), d["A_log"], H, z=d["z"][:, t], S=S, S_out=S, **kw)
        assert S2 is S
        outs.append(y[:, None])
    yr, Sr = oracle.selective_heads(*(p[k] for k in NAMES), p["A_log"], H, **{k: p[k] for k in OPT})
    assert rel_err(torch.cat(outs, 1).float().cpu(), yr) <= TOL[io] and rel_err(S.cpu(), Sr) <= TOL_S


def test_offsets_past_two_to_the_31(lr):  # noqa: F811
    """8192 value channels a step and 2 x 270,001 steps in rows that lie 8448 apart."""
    B, L, H, P, N = 2, 270001, 64, 128, 32
    gen = torch.Generator(device="cuda").manual_seed(5)
    xbc = torch.empty(B, L, H * P + 2 * N + 192, dtype=torch.bfloat16, device="cuda")
    for i in range(0, L, 30000):
        xbc[:, i:i + 30000] = torch.randn(B, min(30000, L - i), xbc.shape[-1], generator=gen, device="cuda")
    x, Bm, Cm = xbc[..., :H * P], xbc[..., H * P:H * P + N], xbc[..., H * P + N:H * P + 2 * N]
    dt = torch.randn(B, L, H, generator=gen, device="cuda").bfloat16()
    A_log = torch.linspace(-3.0, 1.0, H, device="cuda")
    y, S = lr.selective_heads(x, dt, Bm, Cm, A_log, H)
    assert lr.status() == lr.LR_OK
    n = 3000   # decays of about exp(-0.03 n): what came before is gone
    for h in (0, H - 1):
        c = slice(h * P, (h + 1) * P)
        yr, Sr = oracle.selective_heads(x[-1:, -n:, c].cpu(), dt[-1:, -n:, h:h + 1].cpu(), Bm[-1:, -n:].cpu(),
                                        Cm[-1:, -n:].cpu(), A_log[h:h + 1].cpu(), 1)
        assert rel_err(y[-1:, -n // 2:, c].float().cpu(), yr[:, -n // 2:]) <= TOL["bf16"]
        assert rel_err(S[-1:, h:h + 1].cpu(), Sr) <= TOL_S
