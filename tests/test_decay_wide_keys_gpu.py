"""bf16 prompts with more than 128 keys a head: the key columns run in parts
whose outputs are summed in fp32 and rounded once, so the tolerances are those of
the narrower heads (states 2e-5, outputs 1e-2; see test_decay_attn_gpu)."""
import pytest
import torch

import oracle
from conftest import rel_err
from selective_state_space_chunked_gb300 import workloads as wl
from test_decay_attn_gpu import TOL, TOL_S, check, cuda, lr  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dk,dv", [(136, 64), (192, 72), (200, 8), (256, 128), (264, 64), (384, 24), (512, 64)])
@pytest.mark.parametrize("L", [64, 129, 700])
def test_head_widths(lr, dk, dv, L):  # noqa: F811
    check(lr, wl.decay_attn_inputs(2, L, 4, dk, dv, seed=dk + L, io="bf16", Hk=2, with_S0=L != 129), "bf16", scale=0.5)


@pytest.mark.parametrize("dk", [192, 256])
def test_ragged_rows_and_what_lies_behind_them(lr, dk):  # noqa: F811
    lens = [300, 0, 1, 128, 129, 400, -3]
    p = wl.decay_attn_inputs(7, 300, 2, dk, 64, seed=2, io="bf16", with_S0=True)
    for b, n in enumerate(lens):
        for name in ("q", "k", "v"):
            p[name][b, max(n, 0):] = float("nan")
    ref = {k: (torch.nan_to_num(t) if k in ("q", "k", "v") else t) for k, t in p.items()}
    d = cuda(p)
    n = torch.tensor(lens, dtype=torch.int32)
    o, S = lr.decay_attn(d["q"], d["k"], d["v"], 2, a_log=d["a_log"], g=d["g"], S0=d["S0"], lens=n.cuda())
    assert lr.status() == lr.LR_OK
    orf, Srf = oracle.decay_attn(ref["q"], ref["k"], ref["v"], 2, a_log=p["a_log"], g=p["g"], S0=p["S0"], lens=n)
    assert rel_err(o.float().cpu(), orf) <= TOL["bf16"] and rel_err(S.cpu(), Srf) <= TOL_S
    for b, n in enumerate(lens):
        assert torch.all(o[b, max(n, 0):] == 0)


@pytest.mark.parametrize("dk", [160, 256])
def test_segments_and_steep_decays(lr, dk):  # noqa: F811
    p = wl.decay_attn_inputs(1, 5000, 2, dk, 64, seed=4, io="bf16", with_S0=True)
    assert lr.lr_decay_attn_workspace_size(1, 5000, 2, 2, dk, 64, lr.LR_BF16) > 2 * 5000 * 2 * 64 * 4
    check(lr, p, "bf16")
    g = p["g"].float()
    g[:, ::97, 0] = -float("inf")
    g[:, 100:300, 1] = -3.0
    p["g"] = g.to(p["g"].dtype)
    check(lr, p, "bf16", lens=[4321])


def test_host_buffers(lr):  # noqa: F811
    p = wl.decay_attn_inputs(2, 500, 2, 192, 64, seed=6, io="bf16", with_S0=True)
    o, S = lr.decay_attn(p["q"], p["k"], p["v"], 2, a_log=p["a_log"], g=p["g"], S0=p["S0"])
    orf, Srf = oracle.decay_attn(p["q"], p["k"], p["v"], 2, a_log=p["a_log"], g=p["g"], S0=p["S0"])
    assert rel_err(o.float(), orf) <= TOL["bf16"] and rel_err(S, Srf) <= TOL_S
