"""Refusals of the selective scan with heads: every call carries an invalid argument
that the host-side checks catch before any CUDA call, so the fake pointers are never
dereferenced.  Runs without a GPU."""
import pytest
import torch

from test_decay_abi_cpu import FAKE, lr  # noqa: F401

SIZES = dict(H=4, G=2, P=64, N=128)
ROWS = dict(x=FAKE, ldx=256, dt=FAKE, lddt=4, Bm=FAKE, ldb=256, Cm=FAKE, ldc=256, z=FAKE, ldz=256, A_log=FAKE,
            dt_bias=FAKE, Dskip=FAKE)
BAD = [(dict(x=None), -1), (dict(dt=None), -1), (dict(Bm=None), -1), (dict(Cm=None), -1), (dict(A_log=None), -1),
       (dict(y=None), -1), (dict(B=-1), -1), (dict(H=0), -1), (dict(G=0), -1), (dict(G=3), -1), (dict(P=0), -1),
       (dict(N=0), -1), (dict(io=2), -1), (dict(ldx=255), -1), (dict(lddt=3), -1), (dict(ldb=248), -1),
       (dict(ldc=248), -1), (dict(ldz=0), -1), (dict(B=1 << 20, H=1 << 20, G=1), -2),
       (dict(H=1 << 16, P=1 << 16, ldx=1 << 32, ldz=1 << 32, lddt=1 << 16), -2), (dict(x=FAKE + 8), -3),
       (dict(dt=FAKE + 2), -3), (dict(z=FAKE + 8), -3), (dict(A_log=FAKE + 4), -3), (dict(Dskip=FAKE + 4), -3),
       (dict(ldx=260), -3), (dict(ldb=257), -3), (dict(ldc=260), -3), (dict(ldz=258), -3), (dict(io=0, ldx=258), -3)]


@pytest.mark.parametrize("kw,code", BAD + [(dict(L=-1), -1), (dict(N=513, ldb=1 << 12, ldc=1 << 12), -2),
                                           (dict(L=1 << 40), -2), (dict(lens=FAKE + 4), -3), (dict(S0=FAKE + 4), -3),
                                           (dict(S_final=FAKE + 4), -3)])
def test_prompt_form(lr, kw, code):  # noqa: F811
    a = dict(**ROWS, lens=FAKE, S0=FAKE, y=FAKE, S_final=FAKE, B=2, L=9, **SIZES, io=1, dt_softplus=1, workspace=None,
             ws_bytes=0, stream=None)
    a.update(kw)
    assert lr.lr_selective_heads_fwd(*a.values()) == code


@pytest.mark.parametrize("kw,code", BAD + [(dict(S_out=None), -1), (dict(S_in=FAKE + 4), -3)])
def test_step_form(lr, kw, code):  # noqa: F811
    a = dict(**ROWS, S_in=FAKE, S_out=FAKE, y=FAKE, B=2, **SIZES, io=1, dt_softplus=1, stream=None)
    a.update(kw)
    assert lr.lr_selective_heads_step(*a.values()) == code


def test_nothing_to_do_and_workspace_sizes(lr):  # noqa: F811
    none = [None, 256, None, 4, None, 256, None, 256, None, 0, None, None, None, None, None, None]
    assert lr.lr_selective_heads_step(*none, 0, 4, 2, 64, 128, 1, 1, None) == 0
    assert lr.lr_selective_heads_workspace_size(1, 0, 2, 2, 64, 64, 1) == 256
    assert lr.lr_selective_heads_workspace_size(1, 9, 3, 2, 64, 64, 1) == 0
    assert lr.lr_selective_heads_workspace_size(1, 9, 2, 2, 64, 513, 1) == 0


def test_helpers_refuse_wrong_shapes_and_types(lr):  # noqa: F811
    t = torch.zeros
    x, dt, bc, a = t(2, 4, 64), t(2, 4, 4), t(2, 4, 32), t(4)
    for bad in (dict(H=3), dict(H=4, G=3), dict(H=4, z=t(2, 4, 63)), dict(H=4, Dskip=t(3)), dict(H=4, dt_bias=t(5)),
                dict(H=4, G=2, S0=t(2, 4, 16, 15)), dict(H=4, lens=t(3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            lr.selective_heads(x, dt, bc, bc, a, **bad)
    for args in ((x, dt[..., :3], bc, bc), (x, dt, bc, bc[..., :16]), (x, dt, bc[:, :3], bc[:, :3]), (x[0], dt, bc, bc)):
        with pytest.raises(ValueError):
            lr.selective_heads(*args, a, 4)
    with pytest.raises(TypeError):
        lr.selective_heads(x, dt, bc.bfloat16(), bc, a, 4)
    with pytest.raises(TypeError):
        lr.selective_heads(x.half(), dt.half(), bc.half(), bc.half(), a, 4)
    with pytest.raises(ValueError):
        lr.selective_heads_step(x[:, 0], dt[:, 0], bc[:, 0], bc[:, 0], a, 4, S=t(2, 4, 16, 31))
