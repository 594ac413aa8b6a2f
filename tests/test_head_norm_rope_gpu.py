"""Norm of the heads of queries and keys with the rotation in the same pass, against the
float64 oracle.

Metric max|gpu - ref| / max|ref|.  fp32: the sum of squares in chains of at most 16 terms
and 5 additions over lanes (21 * 2^-24, half of it in the root), a division, a root and
three products (8 * 2^-24), sine and cosine and their angle (8 * 2^-24 of the larger
partner), the rotation's sum of two (4 * 2^-24): below 40 * 2^-24 < 3e-6.  bf16: the
store's half step of 2^-8 beside that.
"""
import pytest
import torch

import oracle
from conftest import rel_err
from test_decay_attn_gpu import lr  # noqa: F401

pytestmark = pytest.mark.gpu
TOL = {"f32": 3e-6, "bf16": 2.0 ** -8 + 3e-6}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(lead, H, Hk, d, rot, io, seed=0, apart=0, start=0):
    """q and k are slices of one wider tensor."""
    g = torch.Generator().manual_seed(seed)
    wide = (1.5 * torch.randn(*lead, apart + (H + Hk) * d, generator=g)).to(DT[io]).cuda()
    pos = start + torch.randint(-50, 5000, lead, generator=g)
    return dict(q=wide[..., apart:apart + H * d], k=wide[..., apart + H * d:] if Hk else None, H=H, Hk=Hk,
                gamma_q=torch.randn(d, generator=g).cuda(), gamma_k=torch.randn(d, generator=g).cuda(),
                freqs=(10000.0 ** (-torch.arange(rot // 2) / max(rot // 2, 1))).cuda() if rot else None,
                pos=pos.to(torch.int32).cuda())


def check(got, p, io, norm="rms", pairs="halves", eps=1e-6, tol=None):
    for y, x, h, g in ((got[0], p["q"], p["H"], "gamma_q"), (got[1], p["k"], p["Hk"], "gamma_k")):
        if x is None:
            assert y is None
            continue
        ref = oracle.head_norm_rope(x, h, norm, p[g], p["freqs"], p["pos"], pairs, eps)
        assert y.shape == x.shape and rel_err(y.float().cpu(), ref) <= (tol or TOL[io])


# heads on and off vector boundaries, whole, half and odd parts rotated, lanes of every count
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("H,Hk,d,rot", [
    (1, 1, 16, 16), (4, 2, 32, 32), (3, 1, 64, 64), (16, 4, 128, 128), (2, 2, 128, 64), (6, 3, 80, 80), (2, 1, 96, 32),
    (2, 2, 192, 192), (1, 1, 256, 256), (1, 1, 512, 512), (2, 1, 512, 128), (3, 2, 40, 20), (1, 1, 8, 8), (2, 2, 24, 2),
    (3, 3, 33, 32), (5, 1, 7, 4), (2, 1, 1, 0), (2, 1, 2, 2), (1, 1, 511, 510), (1, 1, 300, 250), (4, 0, 64, 64),
    (2, 2, 64, 0), (1, 1, 130, 130),
    # more heads than a block has lanes for
    (100, 20, 128, 128), (70, 9, 64, 32), (3000, 3000, 2, 2), (33, 0, 256, 128)])
def test_head_layouts(lr, io, pairs, H, Hk, d, rot):  # noqa: F811
    p = inputs((2, 5), H, Hk, d, rot, io, seed=d + rot)
    check(lr.head_norm_rope(**p, pairs=pairs), p, io, pairs=pairs)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("norm", ["rms", "l2", "none"])
@pytest.mark.parametrize("lead", [(1,), (7,), (3, 1), (2, 700), (4, 4096)])
def test_norms_and_token_counts(lr, io, norm, lead):  # noqa: F811
    p = inputs(lead, 6, 2, 64, 64, io, seed=len(lead), apart=24)
    check(lr.head_norm_rope(**p, norm=norm, eps=1e-3), p, io, norm, eps=1e-3)
    p.update(gamma_q=None, gamma_k=None)
    check(lr.head_norm_rope(**p, norm=norm), p, io, norm)


@pytest.mark.parametrize("apart", [8, 4, 3])
def test_slices_on_and_off_boundaries(lr, apart):  # noqa: F811
    for io in ("f32", "bf16"):
        p = inputs((3, 9), 2, 1, 32, 32, io, seed=apart, apart=apart)
        check(lr.head_norm_rope(**p), p, io)


def test_far_positions(lr):  # noqa: F811
    """Angles keep their bits: freqs in turns is exact to 7e-16 of it, so that position
    2^31 - 1 turns by 1.5e-6 of a turn too much at most, 1e-5 radians; 2e-5 with the
    rest.  Nearer ones stay within the usual bound."""
    p = inputs((64,), 2, 1, 128, 128, "f32", seed=5)
    p["pos"] = torch.cat([torch.arange(1 << 20, (1 << 20) + 32), torch.arange(-(1 << 20), 32 - (1 << 20))]).cuda()
    check(lr.head_norm_rope(**p), p, "f32")
    p["pos"] = torch.cat([torch.full((32,), 2 ** 31 - 1), torch.full((32,), -2 ** 31)]).cuda()
    check(lr.head_norm_rope(**p), p, "f32", tol=2e-5)
    p["freqs"] = torch.linspace(-1000.0, 1000.0, 64).cuda()   # many turns a position
    p["pos"] = torch.arange(64).cuda()
    check(lr.head_norm_rope(**p), p, "f32")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_in_place_and_given_outputs(lr, io):  # noqa: F811
    p = inputs((50,), 4, 2, 64, 32, io)
    want = lr.head_norm_rope(**p)
    q, k = p["q"].contiguous(), p["k"].contiguous()
    got = lr.head_norm_rope(**dict(p, q=q, k=k), out=(q, k))
    assert got[0] is q and got[1] is k and torch.equal(q, want[0]) and torch.equal(k, want[1])
    with pytest.raises(ValueError):
        lr.head_norm_rope(**p, out=(q[:10], k))
    empty = dict(p, q=q[:0], k=k[:0], pos=p["pos"][:0])
    assert lr.head_norm_rope(**empty)[0].shape == (0, 256)


def test_infinities_and_nan_stay_in_their_head_and_pair(lr):  # noqa: F811
    p = inputs((3,), 4, 1, 64, 32, "f32")
    want = lr.head_norm_rope(**p, norm="none")
    rms = lr.head_norm_rope(**p)
    q = p["q"].contiguous()
    q[1, 64 + 40] = float("inf")      # head 1, past the rotated part
    q[2, 5] = float("nan")            # head 0, pair 5
    got = lr.head_norm_rope(**dict(p, q=q), norm="none")[0]
    hit = torch.zeros_like(q, dtype=torch.bool)
    hit[1, 64 + 40] = hit[2, 5] = hit[2, 5 + 16] = True
    assert torch.equal(got[~hit], want[0][~hit]) and not torch.isfinite(got[hit]).any()
    got = lr.head_norm_rope(**dict(p, q=q))[0]
    hit[1, 64:128] = hit[2, :64] = True
    assert torch.equal(got[~hit], rms[0][~hit])
    assert torch.isnan(got[1, 64 + 40]) and torch.isnan(got[2, :64]).all()


def test_another_stream_and_a_graph(lr):  # noqa: F811
    p = inputs((9,), 4, 2, 128, 128, "bf16")
    want = lr.head_norm_rope(**p)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        got = lr.head_norm_rope(**p)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_past_2_31_elements(lr):  # noqa: F811
    n, H, d = 1100000, 16, 128
    q = torch.zeros(n, H * d, dtype=torch.bfloat16, device="cuda")
    q[-3:] = torch.randn(3, H * d, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    pos = torch.arange(n, device="cuda")
    f = (10000.0 ** (-torch.arange(64) / 64)).cuda()
    y, _ = lr.head_norm_rope(q, None, H, freqs=f, pos=pos)
    ref = oracle.head_norm_rope(q[-3:], H, "rms", None, f, pos[-3:])
    assert rel_err(y[-3:].float().cpu(), ref) <= TOL["bf16"] and not y[:-3].any()
