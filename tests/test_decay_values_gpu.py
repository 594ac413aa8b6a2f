"""Values at the edges of the decayed linear attention, in steps that belong to a
row, against the float64 oracle: infinities and NaN, values whose scaled form
leaves fp32, and slow steps behind many resets.  Tolerances of finite values: see
test_decay_attn_gpu; that a value is finite, and in the state whether it is an
infinity and of which sign, has no tolerance."""
import numpy as np
import pytest
import torch

import oracle
from selective_state_space_chunked_gb300 import workloads as wl
from test_decay_attn_gpu import TOL, TOL_S, check, cuda, lr  # noqa: F401

pytestmark = pytest.mark.gpu


def same_values(lr, p, io, lens=None, kinds=True):  # noqa: F811
    d = cuda(p)
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    o, S = lr.decay_attn(d["q"], d["k"], d["v"], p["H"], Hk=p["Hk"], a_log=d["a_log"], g=d["g"], S0=d["S0"],
                         lens=None if n is None else n.cuda())
    assert lr.status() == lr.LR_OK
    orf, Srf = oracle.decay_attn(p["q"], p["k"], p["v"], p["H"], Hk=p["Hk"], a_log=p["a_log"], g=p["g"], S0=p["S0"],
                                 lens=n)
    for got, want, tol, exact in ((o.double().cpu().numpy(), orf, TOL[io], False),
                                  (S.double().cpu().numpy(), Srf, TOL_S, kinds)):
        finite = np.isfinite(want)
        assert np.array_equal(np.isfinite(got), finite)
        if finite.any():
            assert np.max(np.abs(got[finite] - want[finite])) <= tol * np.max(np.abs(want[finite]))
        if exact:
            assert np.array_equal(got[~finite], want[~finite], equal_nan=True)
    return o, S


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 200])
@pytest.mark.parametrize("which", ["q", "k", "v"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_bad_value_reaches_no_earlier_step(lr, io, d, which, value):  # noqa: F811
    """One channel of one step in the middle of a chunk."""
    p = wl.decay_attn_inputs(2, 300, 2, d, 64, seed=5, io=io, with_S0=True)
    p[which][0, 200, 3] = value
    o, _ = same_values(lr, p, io)
    assert torch.isfinite(o[0, :200]).all() and torch.isfinite(o[1]).all()
    assert not torch.isfinite(o[0, 200, 3])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 136])
@pytest.mark.parametrize("L", [5, 47, 48, 129])
def test_bad_values_at_the_ends(lr, io, d, L):  # noqa: F811
    for t in (0, L - 1):
        p = wl.decay_attn_inputs(1, L, 3, d, 72, seed=L, io=io)
        p["v"][0, t, 72 + 71] = -float("inf")
        p["v"][0, t, 72 + 5] = float("nan")
        same_values(lr, p, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 192])
def test_bad_values_in_segments(lr, io, d):  # noqa: F811
    """In the state that one segment hands to the next: with slow decays, and with
    decays that leave nothing of a finite state (a NaN stays one)."""
    L = 5000
    p = wl.decay_attn_inputs(1, L, 2, d, 64, seed=6, io=io, decay="head", with_S0=True)
    assert lr.lr_decay_attn_workspace_size(1, L, 2, 2, d, 64, lr.LR_BF16 if io == "bf16" else lr.LR_F32) > 256
    p["a_log"] = torch.full((2,), -2.0 ** -9)
    p["v"][0, 777, 3], p["v"][0, 4999, 70], p["k"][0, 2500, d + 1] = float("inf"), float("nan"), -float("inf")
    same_values(lr, p, io)
    p["a_log"] = torch.tensor([-0.5, -2.0 ** -9])
    same_values(lr, p, io, kinds=False)
    p["S0"][0, 1, 9, 2] = float("nan")
    same_values(lr, p, io, lens=[4321], kinds=False)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_bad_values_with_steep_decays_and_lengths(lr, io, d):  # noqa: F811
    L = 400
    p = wl.decay_attn_inputs(3, L, 2, d, 64, seed=7, io=io, with_S0=True)
    p["S0"][0, 0, 5] = float("nan")
    p["S0"][1, 1, 6, 7] = float("inf")
    p["v"][2, 260, 64 + 9] = float("inf")
    g = p["g"].float()
    g[:, 100:250, 0] = -3.0
    g[:, 300, 1] = -float("inf")   # 0 times an infinity
    p["g"] = g.to(p["g"].dtype)
    same_values(lr, p, io, kinds=False)
    _, S = same_values(lr, p, io, lens=[0, 290, 261], kinds=False)
    assert torch.equal(torch.nan_to_num(S[0].cpu(), 7.0), torch.nan_to_num(p["S0"][0], 7.0))


@pytest.mark.parametrize("d", [64, 128, 160])
@pytest.mark.parametrize("e", [60, 90, 110])
def test_values_far_from_one(lr, d, e):  # noqa: F811
    """bf16 prompts: v of 2^e, where the weights of a chunk reach 2^48."""
    p = wl.decay_attn_inputs(1, 500, 2, d, 64, seed=8, io="bf16", decay="head", with_S0=True)
    p["a_log"] = torch.tensor([-0.1, -0.003])
    p["v"], p["S0"] = p["v"] * 2.0 ** e, p["S0"] * 2.0 ** e
    check(lr, p, "bf16")


def test_slow_steps_behind_many_resets(lr):  # noqa: F811
    """100 resets, then slow steps, in one chunk.  One step has a value and q.k = 1,
    so o_t is the decay factor alone, rounded to bf16 once as a score (the store
    changes nothing more): the rounding of a factor within 2^-14 of the exact one."""
    B, H, L = 4, 8, 128
    q = torch.zeros(B, L, H * 64)
    q[..., ::64] = 1.0
    v = torch.zeros(B, L, H * 64)
    v[:, 100] = 1.0
    gen = torch.Generator().manual_seed(1)
    g = -0.05 * torch.rand(B, L, H, generator=gen)
    g[:, :100] = -float("inf")
    p = {"q": q.bfloat16(), "k": q.bfloat16(), "v": v.bfloat16(), "g": g.bfloat16(), "a_log": None, "S0": None,
         "H": H, "Hk": H}
    o, _ = check(lr, p, "bf16")
    want, _ = oracle.decay_attn(p["q"], p["k"], p["v"], H, g=p["g"])
    low, high = (torch.tensor(want * (1 + e)).bfloat16() for e in (-2.0 ** -14, 2.0 ** -14))
    o = o.cpu()
    assert torch.all((low <= o) & (o <= high))
