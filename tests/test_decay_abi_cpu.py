"""Refusals of the decayed linear attention and the group norm: every call
carries an invalid argument that the host-side checks catch before any CUDA
call, so the fake pointers are never dereferenced.  Runs without a GPU."""
import pytest
import torch

FAKE = 0x7F0000000000


@pytest.fixture(scope="module")
def lr():
    from selective_state_space_chunked_gb300 import build
    build.build()
    from selective_state_space_chunked_gb300 import binding
    return binding


def attn(lr, fn="lr_decay_attn_fwd", **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, a_log=FAKE, g=FAKE, lens=FAKE, scale=1.0, S0=FAKE, o=FAKE, S_final=FAKE,
             B=2, L=64, H=4, Hk=2, dk=128, dv=128, io=1, workspace=None, ws_bytes=0, stream=None)
    a.update(kw)
    if fn != "lr_decay_attn_fwd":
        del a["lens"]
    return getattr(lr, fn)(*a.values())


BAD = [(dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(o=None), -1), (dict(B=-1), -1),
       (dict(L=-1), -1), (dict(H=0), -1), (dict(Hk=0), -1), (dict(Hk=3), -1), (dict(dk=0), -1), (dict(dv=0), -1),
       (dict(io=2), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
       (dict(dk=513), -2), (dict(L=1 << 40), -2), (dict(B=1 << 20, H=1 << 20, Hk=1), -2),
       (dict(q=FAKE + 8), -3), (dict(a_log=FAKE + 4), -3), (dict(g=FAKE + 2), -3), (dict(S_final=FAKE + 4), -3)]


@pytest.mark.parametrize("kw,code", BAD + [(dict(lens=FAKE + 4), -3)])
def test_prompt_form(lr, kw, code):
    assert attn(lr, **kw) == code


@pytest.mark.parametrize("fn", ["lr_decay_attn_fwd_host", "lr_decay_attn_fwd_host_async"])
@pytest.mark.parametrize("kw,code", BAD)
def test_host_forms(lr, fn, kw, code):
    assert attn(lr, fn, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(S_out=None), -1), (dict(o=None), -1), (dict(B=-1), -1), (dict(Hk=3), -1),
    (dict(dk=0), -1), (dict(io=9), -1), (dict(scale=float("nan")), -1), (dict(S_in=FAKE + 4), -3),
    (dict(g=FAKE + 2), -3)])
def test_step_form(lr, kw, code):
    a = dict(q=FAKE, k=FAKE, v=FAKE, a_log=FAKE, g=FAKE, scale=1.0, S_in=FAKE, S_out=FAKE, o=FAKE, B=2, H=4, Hk=2,
             dk=128, dv=128, io=1, stream=None)
    a.update(kw)
    assert lr.lr_decay_attn_step(*a.values()) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(y=None), -1), (dict(N=-1), -1), (dict(C=-1), -1), (dict(G=0), -1), (dict(G=3), -1),
    (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(act=5), -1), (dict(io=3), -1),
    (dict(N=1 << 33), -2), (dict(x=FAKE + 8), -3), (dict(gamma=FAKE + 4), -3), (dict(z=FAKE + 2), -3)])
def test_group_norm(lr, kw, code):
    a = dict(x=FAKE, z=FAKE, gamma=FAKE, beta=FAKE, y=FAKE, N=2, C=64, G=2, eps=1e-5, act=1, io=1, stream=None)
    a.update(kw)
    assert lr.lr_group_norm_act(*a.values()) == code


def test_nothing_to_do_needs_no_pointer(lr):
    assert lr.lr_group_norm_act(None, None, None, None, None, 0, 64, 2, 1e-5, 0, 1, None) == 0
    assert lr.lr_decay_attn_step(None, None, None, None, None, 1.0, None, None, None, 0, 4, 2, 64, 64, 1, None) == 0


def test_workspace_sizes(lr):
    assert lr.lr_decay_attn_workspace_size(1, 0, 2, 2, 64, 64, 1) == 256
    assert lr.lr_decay_attn_workspace_size(0, 9, 2, 2, 64, 64, 1) == 256
    assert lr.lr_decay_attn_workspace_size(1, 9, 3, 2, 64, 64, 1) == 0
    assert lr.lr_decay_attn_workspace_size(1, 9, 2, 2, 513, 64, 1) == 0
    assert lr.lr_decay_attn_fwd_host_workspace_size(0, 9, 2, 2, 64, 64, 1) == 0
    assert lr.lr_decay_attn_fwd_host_workspace_size(1, 9, 3, 2, 64, 64, 1) == 0


def test_helpers_refuse_wrong_shapes_and_types(lr):
    t = torch.zeros
    q = t(2, 4, 64)
    for bad in (dict(H=3), dict(H=4, Hk=3), dict(H=2, g=t(2, 4, 3)), dict(H=2, a_log=t(3)),
                dict(H=2, S0=t(2, 2, 32, 31)), dict(H=2, lens=t(3))):
        with pytest.raises(ValueError):
            lr.decay_attn(q, q, q, **bad)
    with pytest.raises(ValueError):
        lr.decay_attn(q, t(2, 4, 32), q, 2)
    with pytest.raises(TypeError):
        lr.decay_attn(q, q.bfloat16(), q, 2)
    with pytest.raises(TypeError):
        lr.decay_attn(q.half(), q.half(), q.half(), 2)
    with pytest.raises(ValueError):
        lr.decay_attn_step(q[:, 0], q[:, 0], q[:, 0], 2, S=t(2, 2, 32, 30))
    for bad in (dict(G=3), dict(G=2, gamma=t(63)), dict(G=2, z=t(2, 4, 63)), dict(G=2, act="tanh")):
        with pytest.raises(ValueError):
            lr.group_norm_act(q, **bad)
    with pytest.raises(TypeError):
        lr.group_norm_act(q, 2, z=q.bfloat16())
