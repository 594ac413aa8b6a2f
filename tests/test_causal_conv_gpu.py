"""Short causal convolution (prompt and single-token forms) against the float64 oracle.

Metric max|gpu - ref| / max|ref|.  fp32: a sum of at most five terms, each rounded to
2^-24, of a size of up to three times the largest output, and silu to four units in
the last place: 15 * 2^-24 + 4 * 2^-23 < 2e-6.  bf16: the store's half step of 2^-8
beside that.  States are copies of inputs: equal.
"""
import numpy as np
import pytest
import torch

import oracle
from conftest import rel_err
from test_decay_attn_gpu import lr  # noqa: F401

pytestmark = pytest.mark.gpu
TOL = {"f32": 2e-6, "bf16": 2.0 ** -8 + 2e-6}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(B, L, C, W, io, seed=0, apart=0, after=0, state=True, bias=True):
    """x is columns apart .. apart + C of a wider tensor."""
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn(B, L, apart + C + after, generator=g).to(DT[io])
    return dict(x=wide.cuda()[..., apart:apart + C], w=(torch.rand(C, W, generator=g) - 0.5).cuda(),
                bias=torch.randn(C, generator=g).cuda() if bias else None,
                state=torch.randn(B, W - 1, C, generator=g).to(DT[io]).cuda() if state else None)


def check(got, p, io, act="silu", lens=None):
    y, new = got
    yr, nr = oracle.causal_conv(p["x"], p["w"], p["bias"], p["state"], lens, act)
    assert rel_err(y.float().cpu(), yr) <= TOL[io]
    np.testing.assert_array_equal(new.double().cpu().numpy(), nr)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,L,C", [(1, 1, 8), (2, 2, 24), (3, 3, 64), (2, 7, 40), (1, 8, 16), (2, 9, 129), (3, 63, 1),
                                   (1, 64, 264), (2, 65, 33), (5, 200, 72), (2, 1111, 136), (1, 5000, 5), (300, 3, 31),
                                   (40, 300, 520)])
def test_sizes(lr, io, W, B, L, C):  # noqa: F811
    for state, bias, act in ((True, True, "silu"), (False, False, "none")):
        p = inputs(B, L, C, W, io, seed=L + C, state=state, bias=bias)
        check(lr.causal_conv(**p, act=act), p, io, act)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("apart,C,after", [(16, 64, 8), (8, 64, 3), (5, 64, 0), (0, 64, 1), (24, 33, 7), (4, 40, 4)])
def test_slices_of_a_wider_tensor(lr, io, apart, C, after):  # noqa: F811
    """Rows that lie apart, on and off vector boundaries; a slice off a 16-byte
    boundary is copied."""
    p = inputs(3, 50, C, 4, io, seed=C, apart=apart, after=after)
    check(lr.causal_conv(**p), p, io)
    q = dict(p, x=p["x"][:, 20:21], state=p["state"])
    check(lr.causal_conv(**q), q, io)
    one = dict(p, x=p["x"][:, 7])
    y, new = lr.causal_conv_step(**one)
    check((y[:, None], new), dict(one, x=one["x"][:, None]), io)


def test_views_without_even_rows_are_copied(lr):  # noqa: F811
    p = inputs(4, 30, 16, 3, "f32")
    for x in (p["x"][::2, :, :], p["x"][:, ::3], p["x"].transpose(0, 1).contiguous().transpose(0, 1),
              p["x"][:1].expand(4, 30, 16), p["x"][:, :, ::2]):
        q = dict(x=x, w=p["w"][:x.shape[-1]], bias=None, state=None)
        check(lr.causal_conv(**q), q, "f32")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("C", [64, 37])
@pytest.mark.parametrize("W", [2, 4])
def test_ragged_rows(lr, io, C, W):  # noqa: F811
    """Lengths of zero, fewer steps than taps, and beyond the tensor; what stands past
    a length (NaN) reaches neither outputs nor state."""
    L = 133
    lens = [0, 1, 2, 3, 4, 64, 65, 100, L, L + 9, -5]
    p = inputs(len(lens), L, C, W, io, seed=4)
    p["x"] = p["x"].clone()
    for b, n in enumerate(lens):
        p["x"][b, max(n, 0):] = float("nan")
    y, new = lr.causal_conv(**p, lens=torch.tensor(lens).cuda())
    check((y, new), p, io, lens=lens)
    for b, n in enumerate(lens):
        assert torch.all(y[b, max(n, 0):] == 0)
    assert torch.equal(new[0], p["state"][0])
    S = p["state"].clone()   # in place: rows shorter than the taps keep inputs of the old state
    _, same = lr.causal_conv(**dict(p, state=S), lens=torch.tensor(lens).cuda(), out=(torch.empty_like(y), S))
    assert same is S and torch.equal(S, new)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("C,W", [(72, 4), (5, 3), (16, 2)])
def test_pieces_steps_and_states_in_place(lr, io, C, W):  # noqa: F811
    """A prompt, a second piece and tokens, the state in one buffer, equal one call."""
    L = 90
    p = inputs(3, L, C, W, io, seed=9)
    whole, end = lr.causal_conv(**p)
    kw = dict(w=p["w"], bias=p["bias"])
    S = p["state"].clone()
    parts = []
    for a, b in ((0, 1), (1, 3), (3, 80)):
        y = torch.empty(3, b - a, C, dtype=whole.dtype, device="cuda")
        got = lr.causal_conv(p["x"][:, a:b], state=S, out=(y, S), **kw)
        assert got[0] is y and got[1] is S
        parts.append(y)
    for t in range(80, L):
        y, same = lr.causal_conv_step(p["x"][:, t], state=S, state_out=S, **kw)
        assert same is S
        parts.append(y[:, None])
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(S, end)
    short = lr.causal_conv(p["x"][:, :0], state=S, **kw)
    assert short[0].shape == (3, 0, C) and torch.equal(short[1], S)
    assert not lr.causal_conv(p["x"][:, :0], **kw)[1].any()


def test_infinities_and_nan_stay_where_they_are_inputs(lr):  # noqa: F811
    p = inputs(1, 40, 16, 4, "f32", state=False)
    clean, _ = lr.causal_conv(**p, act="none")
    x = p["x"].clone()
    x[0, 10, 3], x[0, 20, 5] = float("nan"), float("inf")
    y, _ = lr.causal_conv(**dict(p, x=x), act="none")
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[0, 10:14, 3] = hit[0, 20:24, 5] = True
    assert torch.equal(y[~hit], clean[~hit]) and not torch.isfinite(y[hit]).any()


def test_another_stream_and_a_graph(lr):  # noqa: F811
    p = inputs(4, 33, 48, 4, "bf16")
    want = lr.causal_conv(**p)
    w1 = lr.causal_conv_step(**dict(p, x=p["x"][:, 0]))
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        got = lr.causal_conv(**p)
        g1 = lr.causal_conv_step(**dict(p, x=p["x"][:, 0]))
    for _ in range(2):
        for t in (*got, *g1):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*got, *g1), (*want, *w1)):
            assert torch.equal(a, b)


def test_past_2_31_elements(lr):  # noqa: F811
    """Offsets past 32 bits: the last row against the oracle."""
    B, L, C = 3, 200000, 4096
    x = torch.zeros(B, L, C, dtype=torch.bfloat16, device="cuda")
    x[-1, -50:] = torch.randn(50, C, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    w = torch.rand(C, 4, generator=torch.Generator().manual_seed(2)).cuda()
    y, new = lr.causal_conv(x, w)
    yr, _ = oracle.causal_conv(x[-1:, -60:], w)
    assert rel_err(y[-1:, -50:].float().cpu(), yr[:, -50:]) <= TOL["bf16"]
    assert torch.equal(new[-1], x[-1, -3:]) and not y[-1, :-50].any() and not y[0].any()
