"""The float64 oracle of the decayed linear attention and of the group norm
with an activation, pinned to closed forms and library routines (CPU)."""
import numpy as np
import pytest
import torch

import oracle


def _rand(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


def test_no_decay_is_causal_linear_attention():
    B, L, H, d = 2, 17, 3, 5
    q, k, v = (_rand(B, L, H * d, seed=s) for s in (1, 2, 3))
    o, S = oracle.decay_attn(q, k, v, H, scale=0.5)
    qh, kh, vh = (t.reshape(B, L, H, d).transpose(0, 2, 1, 3) for t in (q, k, v))
    want = 0.5 * np.tril(qh @ kh.transpose(0, 1, 3, 2)) @ vh
    np.testing.assert_allclose(o.reshape(B, L, H, d).transpose(0, 2, 1, 3), want, atol=1e-12)
    np.testing.assert_allclose(S, vh.transpose(0, 1, 3, 2) @ kh, atol=1e-12)


def test_decay_mask_form_and_shared_key_heads():
    """o = (Q K^T . exp(cumulative log decay differences)) V + decayed S0 part."""
    B, L, H, Hk, dk, dv = 2, 13, 4, 2, 6, 3
    q, k, v = _rand(B, L, Hk * dk, seed=1), _rand(B, L, Hk * dk, seed=2), _rand(B, L, H * dv, seed=3)
    a_log, g = -np.abs(_rand(H, seed=4)) / 10, -np.abs(_rand(B, L, H, seed=5))
    S0 = _rand(B, H, dv, dk, seed=6)
    o, S = oracle.decay_attn(q, k, v, H, Hk=Hk, a_log=a_log, g=g, S0=S0, scale=0.3)
    for b in range(B):
        for h in range(H):
            j = h // (H // Hk)
            qq, kk = q[b, :, j * dk:(j + 1) * dk], k[b, :, j * dk:(j + 1) * dk]
            vv = v[b, :, h * dv:(h + 1) * dv]
            c = np.cumsum(a_log[h] + g[b, :, h])
            D = np.tril(np.exp(np.minimum(c[:, None] - c[None, :], 0.0)))
            want = 0.3 * ((qq @ kk.T * D) @ vv + np.exp(c)[:, None] * (qq @ S0[b, h].T))
            np.testing.assert_allclose(o[b, :, h * dv:(h + 1) * dv], want, atol=1e-12)
            np.testing.assert_allclose(
                S[b, h], (vv * np.exp(c[-1] - c)[:, None]).T @ kk + np.exp(c[-1]) * S0[b, h], atol=1e-12)


def test_equals_hgrn2_with_a_gate_shared_by_the_channels():
    B, L, H, d = 1, 9, 2, 4
    q, k, v = (_rand(B, L, H * d, seed=s) for s in (1, 2, 3))
    g = -np.abs(_rand(B, L, H, seed=4))
    o, S = oracle.decay_attn(q, k, v, H, g=g)
    o2, S2 = oracle.hgrn2(q, k, v, np.repeat(np.exp(g), d, axis=-1), H)
    np.testing.assert_allclose(o, o2, atol=1e-13)
    np.testing.assert_allclose(S, S2, atol=1e-13)


def test_lengths_reset_and_resume():
    B, L, H, d = 3, 10, 2, 4
    q, k, v = (_rand(B, L, H * d, seed=s) for s in (1, 2, 3))
    g = -np.abs(_rand(B, L, H, seed=4))
    S0 = _rand(B, H, d, d, seed=5)
    o, S = oracle.decay_attn(q, k, v, H, g=g, S0=S0, lens=[0, 4, 10])
    assert np.all(o[0] == 0) and np.all(o[1, 4:] == 0)
    np.testing.assert_array_equal(S[0], S0[0])
    o1, S1 = oracle.decay_attn(q[1:2, :4], k[1:2, :4], v[1:2, :4], H, g=g[1:2, :4], S0=S0[1:2])
    np.testing.assert_array_equal(o[1, :4], o1[0])
    np.testing.assert_array_equal(S[1], S1[0])
    o2, S2 = oracle.decay_attn(q[2:, :6], k[2:, :6], v[2:, :6], H, g=g[2:, :6], S0=S0[2:])
    o3, S3 = oracle.decay_attn(q[2:, 6:], k[2:, 6:], v[2:, 6:], H, g=g[2:, 6:], S0=S2)
    np.testing.assert_allclose(np.concatenate([o2, o3], 1), o[2:], atol=1e-13)
    np.testing.assert_allclose(S3, S[2:], atol=1e-13)
    g[:, 5] = -np.inf                            # a reset: the steps before it no longer matter
    o4, _ = oracle.decay_attn(q, k, v, H, g=g, S0=S0)
    o5, _ = oracle.decay_attn(q[:, 5:], k[:, 5:], v[:, 5:], H, g=g[:, 5:])
    np.testing.assert_allclose(o4[:, 5:], o5, atol=1e-13)


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("gate", [True, False])
def test_group_norm_matches_torch(act, gate):
    x, z = torch.randn(7, 24, dtype=torch.float64), torch.randn(7, 24, dtype=torch.float64)
    gamma, beta = torch.randn(24, dtype=torch.float64), torch.randn(24, dtype=torch.float64)
    want = torch.nn.functional.group_norm(x, 4, gamma, beta, 1e-3)
    if act == "silu":
        want = torch.nn.functional.silu(want)
    if gate:
        want = want * torch.nn.functional.silu(z)
    got = oracle.group_norm_act(x, 4, gamma, beta, z if gate else None, act, 1e-3)
    np.testing.assert_allclose(got, want.numpy(), atol=1e-12)
