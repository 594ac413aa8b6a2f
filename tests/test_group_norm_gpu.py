"""Group norm with an activation and a gate against the float64 oracle.

Metric max|gpu - ref| / max|ref|.  fp32: sums of up to 8192 values and one
division, within 5e-6; bf16: the store rounds to 2^-9, 4e-3.  A mean that is m
times the spread costs m roundings of 2^-24 of the centred values.
"""
import pytest
import torch

import oracle
from conftest import rel_err

pytestmark = pytest.mark.gpu
TOL = {"f32": 5e-6, "bf16": 4e-3}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def lr():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_chunked_gb300 import build
    build.build()
    from selective_state_space_chunked_gb300 import binding
    return binding


def inputs(N, C, io, seed=0):
    g = torch.Generator().manual_seed(seed)
    x, z = torch.randn(N, C, generator=g), torch.randn(N, C, generator=g)
    gamma, beta = 1 + 0.2 * torch.randn(C, generator=g), 0.2 * torch.randn(C, generator=g)
    return (1.5 * x + 0.3).to(DT[io]), z.to(DT[io]), gamma, beta


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("N,G,d", [
    (1, 1, 128), (8, 16, 128), (300, 16, 128), (37, 24, 80), (5, 3, 33), (64, 4, 64), (65, 2, 32), (3, 8, 16),
    (7, 5, 8), (9, 7, 4), (2, 1, 4096), (3, 2, 1000), (130, 1, 2048), (4, 1, 8192), (11, 3, 100), (1, 2, 1),
    (6, 1, 7), (33, 2, 500), (5, 1, 5001), (1000, 2, 256), (2, 1, 20000)])
def test_sizes(lr, io, N, G, d):
    x, z, gamma, beta = inputs(N, G * d, io, seed=N + d)
    for act, gate, affine in (("none", True, True), ("silu", False, True), ("silu", True, False),
                              ("none", False, False)):
        ga, be, zz = (gamma, beta, z)
        y = lr.group_norm_act(x.cuda(), G, gamma=ga.cuda() if affine else None, beta=be.cuda() if affine else None,
                              z=zz.cuda() if gate else None, act=act)
        want = oracle.group_norm_act(x, G, ga if affine else None, be if affine else None, zz if gate else None, act)
        assert rel_err(y.float().cpu(), want) <= TOL[io], (act, gate, affine)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [128, 100, 2048])
def test_gamma_or_beta_alone_and_three_axes(lr, io, d):
    x, z, gamma, beta = inputs(12, 2 * d, io, seed=1)
    for ga, be in ((gamma, None), (None, beta)):
        y = lr.group_norm_act(x.cuda().reshape(3, 4, 2 * d), 2, gamma=None if ga is None else ga.cuda(),
                              beta=None if be is None else be.cuda(), z=z.cuda().reshape(3, 4, 2 * d), eps=1e-2)
        assert y.shape == (3, 4, 2 * d)
        want = oracle.group_norm_act(x, 2, ga, be, z, eps=1e-2)
        assert rel_err(y.float().cpu().reshape(12, -1), want) <= TOL[io]


@pytest.mark.parametrize("d", [128, 100, 1024])
def test_a_large_mean_does_not_cancel(lr, d):
    x, _, _, _ = inputs(20, 2 * d, "f32", seed=2)
    x = x + 1000.0
    y = lr.group_norm_act(x.cuda(), 2)
    assert rel_err(y.cpu(), oracle.group_norm_act(x, 2)) <= 1000 / 1.5 * 2 ** -23


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [128, 32, 100, 4096])
def test_constant_groups_and_bad_values_stay_in_their_group(lr, io, d):
    x, z, gamma, beta = inputs(6, 3 * d, io, seed=3)
    x[0, :d] = 2.5                       # no spread: n = beta
    x[1, d] = float("nan")
    x[2, 2 * d] = float("inf")
    x[3, :] = 0.0
    y = lr.group_norm_act(x.cuda(), 3, gamma=gamma.cuda(), beta=beta.cuda(), z=z.cuda(), act="silu").float().cpu()
    want = oracle.group_norm_act(x, 3, gamma, beta, z, "silu")
    bad = torch.zeros(6, 3 * d, dtype=torch.bool)
    bad[1, d:2 * d] = True
    bad[2, 2 * d:] = True
    assert torch.all(torch.isnan(y[bad])) and not torch.any(torch.isnan(y[~bad]))
    assert rel_err(y[~bad], torch.tensor(want)[~bad]) <= TOL[io]


@pytest.mark.parametrize("d", [64, 100])
def test_large_arguments_of_silu(lr, d):
    """silu of large values of either sign is the value or 0, not NaN."""
    x, z, gamma, beta = inputs(4, 2 * d, "f32", seed=4)
    z = z * 1000.0
    y = lr.group_norm_act(x.cuda(), 2, gamma=1e4 * gamma.cuda(), z=z.cuda(), act="silu").cpu()
    assert torch.all(torch.isfinite(y))
    assert rel_err(y, oracle.group_norm_act(x, 2, 1e4 * gamma, None, z, "silu")) <= TOL["f32"]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [128, 100, 3000])
def test_in_place_strides_and_another_stream(lr, io, d):
    x, z, gamma, beta = inputs(50, 2 * d, io, seed=5)
    want = oracle.group_norm_act(x, 2, gamma, beta, z)
    wide = torch.zeros(50, 4 * d, dtype=x.dtype, device="cuda")
    wide[:, :2 * d] = x.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = lr.group_norm_act(wide[:, :2 * d], 2, gamma=gamma.cuda(), beta=beta.cuda(), z=z.cuda())
        xi, zi = x.cuda(), z.cuda()
        y2 = lr.group_norm_act(xi, 2, gamma=gamma.cuda(), beta=beta.cuda(), z=zi, out=xi)
        xi2 = x.cuda()
        y3 = lr.group_norm_act(xi2, 2, gamma=gamma.cuda(), beta=beta.cuda(), z=zi, out=zi)
    s.synchronize()
    assert y2 is xi and y3 is zi
    assert torch.equal(y, y2) and torch.equal(y, y3)
    assert rel_err(y.float().cpu(), want) <= TOL[io]


def test_empty(lr):
    x = torch.zeros(0, 64, device="cuda")
    assert lr.group_norm_act(x, 2).shape == (0, 64)


def test_offsets_past_two_to_the_31(lr):
    N, C = 1100000, 2048                 # 2.25e9 elements
    x = torch.empty(N, C, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in range(0, N, 100000):
        x[i:i + 100000] = torch.randn(100000, C, generator=g, device="cuda")
    y = lr.group_norm_act(x, 16, act="silu")
    for sl in (slice(0, 3), slice(N - 3, N)):
        assert rel_err(y[sl].float().cpu(), oracle.group_norm_act(x[sl].cpu(), 16, act="silu")) <= TOL["bf16"]
