"""Selective scan with heads, ragged batches of more blocks than the GPU has SMs: the scan's
kernels may take the rows by falling length, the gates' launch takes them as they come, and
every row's result stays its own.  Tolerances: see test_selective_heads_gpu."""
import pytest
import torch

from selective_state_space_chunked_gb300 import workloads as wl
from test_decay_attn_gpu import cuda, lr  # noqa: F401
from test_selective_heads_gpu import NAMES, check, same_values

pytestmark = pytest.mark.gpu


def lengths(B, L):
    lens = torch.randint(0, L + 1, (B,), generator=torch.Generator().manual_seed(B)).tolist()
    lens[-1], lens[0] = L, lens[B // 2]   # the longest last, and equal lengths
    return lens


# tile count past 152 in each; N past 128 in parts; past 64 rows as they come
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,G,P,N", [(8, 32, 2, 64, 64), (8, 32, 1, 64, 128), (9, 20, 4, 72, 48), (5, 24, 2, 64, 160),
                                       (64, 3, 1, 64, 64), (65, 3, 3, 64, 64), (20, 4, 2, 128, 136)])
def test_rows_in_any_order(lr, io, B, H, G, P, N):  # noqa: F811
    L = 300
    p = wl.selective_heads_inputs(B, L, H, G, P, N, seed=B + N, io=io, with_S0=True)
    lens = lengths(B, L)
    y, S = check(lr, p, io, lens=lens)
    for b, n in enumerate(lens):
        assert torch.all(y[b, n:] == 0)
        if n == 0:
            assert torch.equal(S[b].cpu(), p["S0"][b])


@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("N", [64, 160])
@pytest.mark.parametrize("which", ["x", "Bm", "S0"])
def test_a_bad_value_in_a_middle_row(lr, N, which, z):  # noqa: F811
    """The block that goes through its steps again is the row's own."""
    B, L, H = 8, 200, 24
    p = wl.selective_heads_inputs(B, L, H, 2, 64, N, seed=N, io="bf16", z=z, with_S0=True, rate=(0.1, 1.0))
    lens = [40, 200, 131, 90, 200, 7, 180, 128]
    if which == "S0":
        p["S0"][3, 5, 7, 9] = float("inf")
    else:
        p[which][3, 60, 3] = float("inf")
    y, S = same_values(lr, p, "bf16", lens=lens)
    others = [b for b in range(B) if b != 3]
    assert torch.isfinite(y[others]).all() and torch.isfinite(S[others]).all()
    assert not torch.isfinite(S[3]).all()


def test_rows_of_a_batch_are_those_of_their_own_calls(lr):  # noqa: F811
    """Bit for bit where nothing but the order of the blocks differs."""
    B, L, H, P, N = 8, 384, 32, 64, 64
    p = wl.selective_heads_inputs(B, L, H, 2, P, N, seed=4, io="bf16", with_S0=True)
    d = cuda(p)
    lens = torch.tensor(lengths(B, L), dtype=torch.int32).cuda()
    kw = {k: d[k] for k in ("Dskip", "dt_bias")}
    y, S = lr.selective_heads(*(d[k] for k in NAMES), d["A_log"], H, G=2, lens=lens, z=d["z"], S0=d["S0"], **kw)
    for b in range(B):
        y1, S1 = lr.selective_heads(*(d[k][b:b + 1] for k in NAMES), d["A_log"], H, G=2, lens=lens[b:b + 1],
                                    z=d["z"][b:b + 1], S0=d["S0"][b:b + 1], **kw)
        assert torch.equal(y[b], y1[0]) and torch.equal(S[b], S1[0])
