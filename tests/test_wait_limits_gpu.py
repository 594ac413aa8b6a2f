"""The limit of a kernel's waits is for its own work.  In a call of several launches the last
one starts early, and some of its warps wait for others that wait for the launch before: that
one may take longer than the limit (an infinity sends its block through a segment one step
at a time, 1 us each) without the call failing."""
import pytest
import torch

from selective_state_space_chunked_gb300 import workloads as wl
from test_decay_attn_gpu import lr  # noqa: F401

pytestmark = pytest.mark.gpu
L, H = 32768, 64   # two segments of 16384 steps: 16 ms of single steps


@pytest.fixture
def limit(lr):  # noqa: F811
    def set_ms(ms):
        lr.lr_test_withhold_split(99 if ms else -1, ms or 1000)   # (no scan here has a split 99)
    yield set_ms
    set_ms(None)


def same_under_a_short_limit(lr, limit, call):  # noqa: F811
    want = call()
    assert lr.status() == lr.LR_OK
    torch.cuda.synchronize()
    limit(3)
    got = call()
    assert lr.status() == lr.LR_OK
    for g, w in zip(got, want):
        assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))
    assert not torch.isfinite(want[1]).all()


@pytest.mark.parametrize("N", [64, 192])
def test_selective_heads(lr, limit, N):  # noqa: F811
    p = wl.selective_heads_inputs(1, L, H if N == 64 else H // 2, 1, 64, N, seed=1, io="bf16", z=False,
                                  device="cuda", rate=(1e-4, 1e-3))
    p["x"][0, 5, 3] = float("inf")
    same_under_a_short_limit(lr, limit, lambda: lr.selective_heads(
        p["x"], p["dt"], p["Bm"], p["Cm"], p["A_log"], p["H"], Dskip=p["Dskip"], dt_bias=p["dt_bias"]))


def test_decay_attn(lr, limit):  # noqa: F811
    gen = torch.Generator(device="cuda").manual_seed(2)
    q, k = (torch.randn(1, L, 64, generator=gen, device="cuda").bfloat16() for _ in range(2))
    v = torch.randn(1, L, H * 64, generator=gen, device="cuda").bfloat16()
    v[0, 5, 3] = float("inf")
    a_log = torch.full((H,), -1e-5, device="cuda")
    same_under_a_short_limit(lr, limit, lambda: lr.decay_attn(q, k, v, H, Hk=1, a_log=a_log))
