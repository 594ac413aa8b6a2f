"""The skip of the selective scan with heads is an fp32 parameter and is added in fp32: with
C = 0 an output is Dskip x silu(z), rounded once.

Bound of an output: half a step of its type at the exact value, and the fp32 arithmetic before
it.  fp32 outputs without a gate: that of one product, the rounding itself.  bf16 outputs: the
skip over the row's factor u (a reciprocal, 2 * 2^-24, and a product), times x, times u (a
rounding each), 5 * 2^-24 < 2^-21.  A gate: the exponent's argument is rounded (|z| log2(e)
2^-24 for |z| < 5, 8 * 2^-24 of the power), the power (2 * 2^-24), the sum, the reciprocal
and two products (5 * 2^-24): 15 * 2^-24 more, 2^-19 in all.
"""
import numpy as np
import pytest
import torch

import oracle
from selective_state_space_chunked_gb300 import workloads as wl
from test_decay_attn_gpu import cuda, lr  # noqa: F401

pytestmark = pytest.mark.gpu
NAMES = ("x", "dt", "Bm", "Cm")
BITS = {"f32": 24, "bf16": 8}
FP32 = {"f32": 2.0 ** -24, "bf16": 2.0 ** -21}   # of the arithmetic, without a gate


def half_step(v, io):
    return np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -100))) - BITS[io])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 47, 48, 300])
@pytest.mark.parametrize("N", [64, 128, 160])
@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("steep", [False, True])
def test_skip_is_rounded_with_the_output_alone(lr, io, L, N, z, steep):  # noqa: F811
    H, P = 4, 72
    p = wl.selective_heads_inputs(2, L, H, 2, P, N, seed=L + N, io=io, z=z)
    p["Cm"].zero_()
    if z:
        p["z"] = p["z"].clamp(-5.0, 5.0)
    if steep:
        p["dt"][:, :, :2] = 8.0
    p["Dskip"] = torch.tensor([1.0 + 2.0 ** -8 - 2.0 ** -20, 1.00781, -0.3337, 2.0 ** -9 + 2.0 ** -19])
    d = cuda(p)
    lens = torch.tensor([L, (L + 1) // 2], dtype=torch.int32)
    kw = dict(z=d["z"], Dskip=d["Dskip"], dt_bias=d["dt_bias"])
    y, _ = lr.selective_heads(*(d[k] for k in NAMES), d["A_log"], H, G=2, lens=lens.cuda(), **kw)
    assert lr.status() == lr.LR_OK
    yr, _ = oracle.selective_heads(*(p[k] for k in NAMES), p["A_log"], H, G=2, lens=lens.tolist(), z=p["z"],
                                   Dskip=p["Dskip"], dt_bias=p["dt_bias"])
    off = np.abs(y.double().cpu().numpy() - yr)
    assert np.all(off <= half_step(yr, io) + np.abs(yr) * (2.0 ** -19 if z else FP32[io]))


def test_skip_over_segments_of_a_long_prompt(lr):  # noqa: F811
    """Chunks in turn: the skip's x is that of the output's own step."""
    p = wl.selective_heads_inputs(1, 9000, 2, 1, 64, 64, seed=3, io="bf16", z=False)
    p["Cm"].zero_()
    d = cuda(p)
    y, _ = lr.selective_heads(*(d[k] for k in NAMES), d["A_log"], 2, Dskip=d["Dskip"], dt_bias=d["dt_bias"])
    want = (p["Dskip"].double().numpy()[:, None] * p["x"].double().numpy().reshape(1, 9000, 2, 64)).reshape(1, 9000, 128)
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= half_step(want, "bf16") + np.abs(want) * FP32["bf16"])
