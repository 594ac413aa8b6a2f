"""Rotation by large angles against exact ones: pos freqs is reduced modulo a turn in rational
arithmetic (float64 would lose the angle itself).  The kernel's turn is off by |pos| 2^-64 at
most, nothing beside fp32's own roundings, so the bounds are test_head_norm_rope_gpu's at
every position and frequency."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from conftest import rel_err
from test_decay_attn_gpu import lr  # noqa: F401
from test_head_norm_rope_gpu import DT, TOL

pytestmark = pytest.mark.gpu
TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def rotated(x, freqs, pos, pairs):
    """The heads of x (n, H, d) turned by exact angles."""
    ang = np.array([[float(Fraction(int(p)) * Fraction(float(f)) % TWO_PI) for f in freqs] for p in pos])[:, None]
    m = len(freqs)
    a, b = (slice(0, m), slice(m, 2 * m)) if pairs == "halves" else (slice(0, 2 * m, 2), slice(1, 2 * m, 2))
    y = x.copy()
    y[..., a], y[..., b] = x[..., a] * np.cos(ang) - x[..., b] * np.sin(ang), x[..., b] * np.cos(ang) + x[..., a] * np.sin(ang)
    return y


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("freq", [2.0 ** 20 - 1.0, 777.7, 1.0, 1e-3, 1e-12])
def test_far_positions_and_high_frequencies(lr, io, pairs, freq):  # noqa: F811
    g = torch.Generator().manual_seed(3)
    pos = torch.tensor([0, 1, -1, 12345, 1 << 20, -(1 << 20) + 7, 2 ** 31 - 1, 2 ** 31 - 2, -2 ** 31, 1234567891],
                       dtype=torch.int32)
    freqs = freq * (0.5 + 0.5 * torch.rand(16, generator=g))
    freqs[::3] *= -1
    x = torch.randn(len(pos), 2 * 32, generator=g).to(DT[io])
    q, k = lr.head_norm_rope(x.cuda(), x.cuda(), 2, norm="none", freqs=freqs.cuda(), pos=pos.cuda(), pairs=pairs)
    ref = rotated(x.double().numpy().reshape(-1, 2, 32), freqs.tolist(), pos.tolist(), pairs).reshape(len(pos), 64)
    assert rel_err(q.float().cpu(), ref) <= TOL[io] and torch.equal(q, k)
