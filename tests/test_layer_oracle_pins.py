"""The float64 oracle of the short causal convolution, of the selective scan with heads
and of the norm with rotation of heads, pinned to library routines and closed forms
(CPU)."""
import numpy as np
import pytest
import torch

import oracle


def _rand(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


# ------------------------------------------------------------ convolution
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_convolution_matches_torch(W, act):
    B, L, C = 2, 11, 5
    x, w, bias, state = _rand(B, L, C), _rand(C, W, seed=1), _rand(C, seed=2), _rand(B, W - 1, C, seed=3)
    full = torch.from_numpy(np.concatenate([state, x], 1)).transpose(1, 2)
    want = torch.nn.functional.conv1d(full, torch.from_numpy(w)[:, None], torch.from_numpy(bias), groups=C)
    want = torch.nn.functional.silu(want) if act == "silu" else want
    y, new = oracle.causal_conv(x, w, bias, state, act=act)
    np.testing.assert_allclose(y, want.transpose(1, 2).numpy(), atol=1e-13)
    np.testing.assert_array_equal(new, x[:, L - (W - 1):])


def test_convolution_runs_in_pieces_and_rows_by_their_lengths():
    B, L, C, W = 4, 9, 3, 4
    x, w, state = _rand(B, L, C), _rand(C, W, seed=1), _rand(B, W - 1, C, seed=3)
    lens = [0, 1, 2, 9]
    y, new = oracle.causal_conv(x, w, None, state, lens)
    for b, n in enumerate(lens):
        yb, nb = oracle.causal_conv(x[b:b + 1, :n], w, None, state[b:b + 1])
        np.testing.assert_array_equal(y[b, :n], yb[0])
        assert np.all(y[b, n:] == 0)
        np.testing.assert_array_equal(new[b], np.concatenate([state[b], x[b, :n]])[-(W - 1):])
        np.testing.assert_array_equal(new[b], nb[0])
    whole, end = oracle.causal_conv(x, w)
    a, mid = oracle.causal_conv(x[:, :2], w)
    b, last = oracle.causal_conv(x[:, 2:], w, None, mid)
    np.testing.assert_allclose(np.concatenate([a, b], 1), whole, atol=1e-14)
    np.testing.assert_array_equal(last, end)


# ------------------------------------------------- selective scan with heads
def test_heads_match_the_selective_scan_with_equal_channels():
    """A channel of the selective scan is a head of one value channel: B and C are
    shared by all, and A takes one value for its 16 states."""
    B, L, D = 2, 13, 3
    x, dt, z = _rand(B, L, D), _rand(B, L, D, seed=1) - 2.0, _rand(B, L, D, seed=2)
    Bm, Cm, S0 = _rand(B, L, 16, seed=3), _rand(B, L, 16, seed=4), _rand(B, D, 16, seed=5)
    A_log, skip = np.log(np.array([1.0, 3.0, 7.0])), _rand(D, seed=6)
    y, S = oracle.selective_heads(x, dt, Bm, Cm, A_log, D, z=z, Dskip=skip, S0=S0[:, :, None])
    yr, hr = oracle.selective_scan(x, dt, Bm, Cm, np.repeat(A_log[:, None], 16, 1), z=z, Dskip=skip, h0=S0)
    np.testing.assert_allclose(y, yr, atol=1e-12)
    np.testing.assert_allclose(S[:, :, 0], hr, atol=1e-12)


def test_heads_by_the_recurrence():
    B, L, H, G, P, N = 2, 7, 4, 2, 3, 5
    x, dt, z = _rand(B, L, H * P), _rand(B, L, H, seed=1), _rand(B, L, H * P, seed=2)
    Bm, Cm, S0 = _rand(B, L, G * N, seed=3), _rand(B, L, G * N, seed=4), _rand(B, H, P, N, seed=5)
    A_log, bias, skip = _rand(H, seed=6), _rand(H, seed=7), _rand(H, seed=8)
    lens = [7, 4]
    y, S = oracle.selective_heads(x, dt, Bm, Cm, A_log, H, G, z, skip, bias, S0, lens)
    for b in range(B):
        for h in range(H):
            s, j = S0[b, h].copy(), h // (H // G)
            for t in range(lens[b]):
                delta = np.log1p(np.exp(dt[b, t, h] + bias[h]))
                xt = x[b, t, h * P:(h + 1) * P]
                s = np.exp(-np.exp(A_log[h]) * delta) * s + np.outer(delta * xt, Bm[b, t, j * N:(j + 1) * N])
                zt = z[b, t, h * P:(h + 1) * P]
                want = (s @ Cm[b, t, j * N:(j + 1) * N] + skip[h] * xt) * zt / (1 + np.exp(-zt))
                np.testing.assert_allclose(y[b, t, h * P:(h + 1) * P], want, atol=1e-12)
            np.testing.assert_allclose(S[b, h], s, atol=1e-12)
        assert np.all(y[b, lens[b]:] == 0)


# ---------------------------------------------------------- norm and rotation
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_rotation_is_a_complex_product(pairs):
    n, H, d, rot = 6, 3, 10, 8
    x, freqs, pos = _rand(n, H * d), np.abs(_rand(rot // 2, seed=1)), np.array([0, 1, -4, 77, 5000, 1 << 20])
    y = oracle.head_norm_rope(x, H, "none", None, freqs, pos, pairs).reshape(n, H, d)
    v = x.reshape(n, H, d)
    c = v[..., :rot // 2] + 1j * v[..., rot // 2:rot] if pairs == "halves" else v[..., 0:rot:2] + 1j * v[..., 1:rot:2]
    c = c * np.exp(1j * pos[:, None, None] * freqs)
    got = y[..., :rot // 2] + 1j * y[..., rot // 2:rot] if pairs == "halves" else y[..., 0:rot:2] + 1j * y[..., 1:rot:2]
    np.testing.assert_allclose(got, c, atol=1e-12)
    np.testing.assert_array_equal(y[..., rot:], v[..., rot:])


def test_scores_depend_on_the_distance_alone():
    d, freqs = 16, 10000.0 ** (-np.arange(8) / 8)
    q, k = _rand(1, d), _rand(1, d, seed=1)
    def score(a, b):
        r = [oracle.head_norm_rope(v, 1, "none", None, freqs, np.array([p])) for v, p in ((q, a), (k, b))]
        return float((r[0] * r[1]).sum())
    np.testing.assert_allclose(score(9, 4), score(1009, 1004), atol=1e-11)


def test_norms():
    x, g = _rand(4, 24), _rand(8, seed=1)
    rms = torch.nn.functional.rms_norm(torch.from_numpy(x).reshape(4, 3, 8), (8,), torch.from_numpy(g), 1e-3)
    np.testing.assert_allclose(oracle.head_norm_rope(x, 3, "rms", g, eps=1e-3), rms.reshape(4, 24).numpy(), atol=1e-13)
    v = x.reshape(4, 3, 8)
    l2 = v / np.sqrt((v ** 2).sum(-1, keepdims=True) + 1e-3) * g
    np.testing.assert_allclose(oracle.head_norm_rope(x, 3, "l2", g, eps=1e-3), l2.reshape(4, 24), atol=1e-13)
