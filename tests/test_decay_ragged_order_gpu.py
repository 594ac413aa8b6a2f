"""Ragged batches of few and of many blocks: the kernels may take the rows in
any order, every row's result stays its own.  Tolerances: see test_decay_attn_gpu."""
import pytest
import torch

import oracle
from conftest import rel_err
from selective_state_space_chunked_gb300 import workloads as wl
from test_decay_attn_gpu import TOL, TOL_S, check, cuda, lr  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,dk,dv", [(2, 80, 32, 64), (9, 20, 64, 64), (64, 3, 64, 64), (65, 3, 64, 64), (40, 4, 136, 64)])
def test_rows_in_any_order(lr, io, B, H, dk, dv):  # noqa: F811
    L = 140
    gen = torch.Generator().manual_seed(B)
    lens = torch.randint(0, L + 1, (B,), generator=gen).tolist()
    lens[-1] = L
    lens[0] = lens[B // 2]   # equal lengths
    check(lr, wl.decay_attn_inputs(B, L, H, dk, dv, seed=B, io=io, with_S0=True), io, lens=lens)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_equal_and_empty_rows(lr, io):  # noqa: F811
    p = wl.decay_attn_inputs(6, 100, 40, 64, 64, seed=1, io=io, with_S0=True)
    check(lr, p, io, lens=[100] * 6)
    d = cuda(p)
    o, S = lr.decay_attn(d["q"], d["k"], d["v"], 40, a_log=d["a_log"], g=d["g"], S0=d["S0"],
                         lens=torch.zeros(6, dtype=torch.int32, device="cuda"))
    assert torch.all(o == 0) and torch.equal(S, d["S0"])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_segments_of_ragged_rows(lr, io):  # noqa: F811
    p = wl.decay_attn_inputs(3, 4000, 2, 64, 64, seed=3, io=io, with_S0=True)
    lens = [1700, 4000, 3]
    check(lr, p, io, lens=lens)
    n = torch.tensor(lens, dtype=torch.int32)
    d = cuda(p)
    outs = [lr.decay_attn(d["q"], d["k"], d["v"], 2, a_log=d["a_log"], g=d["g"], S0=d["S0"], lens=n.cuda())
            for _ in range(3)]
    for o, S in outs[1:]:   # the same every time
        assert torch.equal(o, outs[0][0]) and torch.equal(S, outs[0][1])
    orf, Srf = oracle.decay_attn(p["q"], p["k"], p["v"], 2, a_log=p["a_log"], g=p["g"], S0=p["S0"], lens=n)
    assert rel_err(outs[0][0].float().cpu(), orf) <= TOL[io] and rel_err(outs[0][1].cpu(), Srf) <= TOL_S
