"""Refusals of the short causal convolution and of the norm with rotation of heads:
every call carries an invalid argument that the host-side checks catch before any
CUDA call, so the fake pointers are never dereferenced.  Runs without a GPU."""
import pytest
import torch

from test_decay_abi_cpu import FAKE, lr  # noqa: F401


CONV_BAD = [(dict(x=None), -1), (dict(w=None), -1), (dict(y=None), -1), (dict(B=-1), -1), (dict(C=-1), -1),
            (dict(W=1), -1), (dict(ldx=63), -1), (dict(act=2), -1), (dict(io=2), -1), (dict(W=5), -2),
            (dict(C=1 << 40, ldx=1 << 40), -2), (dict(B=1 << 40), -2), (dict(x=FAKE + 8), -3), (dict(w=FAKE + 4), -3),
            (dict(bias=FAKE + 4), -3), (dict(y=FAKE + 2), -3)]


@pytest.mark.parametrize("kw,code", CONV_BAD + [(dict(L=-1), -1), (dict(L=1 << 40), -2), (dict(L=2 ** 31 - 60), -2), (dict(lens=FAKE + 4), -3),
                                                (dict(state=FAKE + 2), -3), (dict(state_out=FAKE + 2), -3)])
def test_convolution(lr, kw, code):  # noqa: F811
    a = dict(x=FAKE, ldx=64, w=FAKE, bias=FAKE, state=FAKE, lens=FAKE, y=FAKE, state_out=FAKE, B=2, L=9, C=64, W=4,
             act=1, io=1, stream=None)
    a.update(kw)
    assert lr.lr_causal_conv_fwd(*a.values()) == code


@pytest.mark.parametrize("kw,code", CONV_BAD + [(dict(state_out=None), -1), (dict(state_in=FAKE + 2), -3)])
def test_convolution_step(lr, kw, code):  # noqa: F811
    a = dict(x=FAKE, ldx=64, w=FAKE, bias=FAKE, state_in=FAKE, state_out=FAKE, y=FAKE, B=2, C=64, W=4, act=1, io=1,
             stream=None)
    a.update(kw)
    assert lr.lr_causal_conv_step(*a.values()) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(q_out=None), -1), (dict(k_out=None), -1), (dict(freqs=None), -1),
    (dict(pos=None), -1), (dict(N=-1), -1), (dict(H=0), -1), (dict(Hk=-1), -1), (dict(d=0), -1), (dict(rot=-2), -1),
    (dict(rot=66), -1), (dict(rot=3), -1), (dict(ldq=255), -1), (dict(ldk=127), -1), (dict(norm=3), -1),
    (dict(norm=-1), -1), (dict(pairs=2), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(io=2), -1),
    (dict(d=513, rot=0), -2), (dict(N=1 << 33), -2), (dict(H=1 << 33), -2), (dict(H=1 << 24, ldq=1 << 30), -2), (dict(q=FAKE + 8), -3),
    (dict(k=FAKE + 8), -3), (dict(gamma_q=FAKE + 4), -3), (dict(freqs=FAKE + 4), -3), (dict(pos=FAKE + 4), -3),
    (dict(k_out=FAKE + 8), -3)])
def test_norm_and_rotation(lr, kw, code):  # noqa: F811
    a = dict(q=FAKE, ldq=256, k=FAKE, ldk=128, gamma_q=FAKE, gamma_k=FAKE, freqs=FAKE, pos=FAKE, q_out=FAKE, k_out=FAKE,
             N=5, H=4, Hk=2, d=64, rot=64, norm=1, eps=1e-6, pairs=0, io=1, stream=None)
    a.update(kw)
    assert lr.lr_head_norm_rope(*a.values()) == code


def test_nothing_to_do_needs_no_pointer(lr):  # noqa: F811
    for B, L, C in ((0, 4, 8), (2, 0, 8), (2, 4, 0)):
        assert lr.lr_causal_conv_fwd(None, C, None, None, None, None, None, None, B, L, C, 4, 1, 1, None) == 0
    assert lr.lr_causal_conv_step(None, 8, None, None, None, None, None, 0, 8, 4, 1, 1, None) == 0
    assert lr.lr_head_norm_rope(None, 64, None, 0, None, None, None, None, None, None, 0, 1, 0, 64, 64, 1, 1e-6, 0, 1,
                                None) == 0


def test_helpers_refuse_wrong_shapes_and_types(lr):  # noqa: F811
    t = torch.zeros
    x, w = t(2, 4, 64), t(64, 4)
    for bad in (dict(bias=t(63)), dict(state=t(2, 4, 64)), dict(act="tanh")):
        with pytest.raises(ValueError):
            lr.causal_conv(x, w, **bad)
        with pytest.raises(ValueError):
            lr.causal_conv_step(x[:, 0], w, **bad)
    for bad in (w[:63], t(64), t(64, 1, 4)):
        with pytest.raises(ValueError):
            lr.causal_conv(x, bad)
    with pytest.raises(ValueError):
        lr.causal_conv(x[0], w)
    with pytest.raises(ValueError):
        lr.causal_conv(x, w, lens=t(3, dtype=torch.int32))
    with pytest.raises(TypeError):
        lr.causal_conv(x, w, lens=t(2))
    with pytest.raises(TypeError):
        lr.causal_conv(x, w, state=t(2, 3, 64).bfloat16())
    with pytest.raises(TypeError):
        lr.causal_conv(x.half(), w)
    f, pos = t(16), t(2, 4, dtype=torch.int32)
    for bad in (dict(H=3), dict(H=2, Hk=3), dict(H=2, gamma_q=t(31)), dict(H=2, freqs=t(17), pos=pos),
                dict(H=2, freqs=f), dict(H=2, freqs=f, pos=pos[:1]), dict(H=2, norm="max"), dict(H=2, pairs="odd")):
        with pytest.raises(ValueError):
            lr.head_norm_rope(x, x, **bad)
    with pytest.raises(TypeError):
        lr.head_norm_rope(x, x.bfloat16(), 2)
    with pytest.raises(TypeError):
        lr.head_norm_rope(x, x, 2, freqs=f, pos=pos.float())
    with pytest.raises(TypeError):
        lr.head_norm_rope(x.half(), None, 2)
