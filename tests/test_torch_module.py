"""The torch helpers' short path: it declines what is not already in the kernels'
form (the helper then converts or refuses), and gives the helper's own results."""
import pytest

torch = pytest.importorskip("torch")

from selective_state_space_chunked_gb300 import workloads as wl  # noqa: E402


@pytest.fixture(scope="module")
def lr():
    from selective_state_space_chunked_gb300 import build
    build.build()
    from selective_state_space_chunked_gb300 import binding
    return binding


def test_host_tensors_and_other_objects_are_declined(lr):
    q, v, S = torch.zeros(2, 8), torch.zeros(2, 8), torch.zeros(2, 2, 4, 4)
    assert lr._lrtorch.decay_attn_step(q, q, v, 2, None, None, None, S, None, 1.0) is None
    assert lr._lrtorch.decay_attn(q[None], q[None], v[None], 2, None, None, None, None, None, 1.0) is None
    assert lr._lrtorch.group_norm_act(q, 2, None, None, None, 0, 1e-5, None) is None
    for bad in (None, 3, "q", object()):
        assert lr._lrtorch.decay_attn_step(bad, q, v, 2, None, None, None, S, None, 1.0) is None
        assert lr._lrtorch.group_norm_act(bad, 2, None, None, None, 0, 1e-5, None) is None
    assert lr._lrtorch.group_norm_act(q) is None   # too few arguments


def _step_args(io="bf16"):
    p = wl.decay_attn_inputs(3, 1, 4, 32, 16, 5, io=io, Hk=2, with_S0=True)
    p = {n: t.cuda() if torch.is_tensor(t) else t for n, t in p.items()}
    return p["q"][:, 0].contiguous(), p["k"][:, 0].contiguous(), p["v"][:, 0].contiguous(), p["a_log"], \
        p["g"][:, 0].contiguous(), p["S0"]


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_the_short_path_gives_the_helpers_results(lr, io, monkeypatch):
    q, k, v, a, g, S = _step_args(io)
    x = torch.randn(7, 64, device="cuda").to(q.dtype)
    p = wl.decay_attn_inputs(2, 90, 4, 32, 16, 6, io=io, Hk=2, with_S0=True)
    p = {n: t.cuda() if torch.is_tensor(t) else t for n, t in p.items()}
    lens = torch.tensor([90, 0], dtype=torch.int32, device="cuda")

    def calls():
        o, Sn = lr.decay_attn_step(q, k, v, 4, Hk=2, a_log=a, g=g, S=S)
        inplace = S.clone()
        _, same = lr.decay_attn_step(q, k, v, 4, Hk=2, a_log=a, g=g, S=inplace, S_out=inplace, scale=2)
        assert same is inplace
        out = torch.empty_like(x)
        assert lr.group_norm_act(x, 4, out=out) is out
        o2, S2 = lr.decay_attn(p["q"], p["k"], p["v"], 4, Hk=2, a_log=p["a_log"], g=p["g"], S0=p["S0"], lens=lens)
        lr.check_status()
        return o, Sn, inplace, out, lr.group_norm_act(x, 4, z=x, act="silu"), o2, S2

    short = calls()
    called = []
    for name in ("decay_attn", "decay_attn_step", "group_norm_act"):
        monkeypatch.setattr(lr._lrtorch, name, lambda *args: called.append(1))
    long = calls()
    assert len(called) == 5
    for s, t in zip(short, long):
        assert torch.equal(s, t)


@pytest.mark.gpu
def test_what_it_takes_and_what_it_declines(lr):
    q, k, v, a, g, S = _step_args()
    take = lambda *args: lr._lrtorch.decay_attn_step(*args)  # noqa: E731
    good = (q, k, v, 4, 2, a, g, S, None, 1.0)
    assert take(*good) is not None
    for i, other in [(0, q.float()), (0, q[:, ::2]), (1, k[:2]), (2, v.cpu()), (2, v[:, :-1].contiguous()), (3, 3),
                     (3, "4"), (4, 3), (5, a.double()), (5, a[:3]), (6, g.float()), (7, S.transpose(2, 3)),
                     (7, S.bfloat16()), (8, S[:, :, :8]), (9, float("nan")), (9, "1")]:
        args = list(good)
        args[i] = other
        assert take(*args) is None, i
    # what is declined is converted, or refused with the reason
    o, _ = lr.decay_attn_step(q, k, v, 4, Hk=2, a_log=a.double(), g=g, S=S)
    assert torch.equal(o, take(*good)[0])
    with pytest.raises(ValueError):
        lr.decay_attn_step(q, k[:2], v, 4, Hk=2)
    with pytest.raises(lr.LrError):
        lr.decay_attn_step(q, k, v, 4, Hk=2, a_log=a, g=g, S=S, scale=float("nan"))


@pytest.mark.gpu
def test_the_call_runs_on_the_current_stream(lr):
    q, k, v, a, g, S = _step_args("f32")
    want, _ = lr.decay_attn_step(q, k, v, 4, Hk=2, a_log=a, g=g, S=S)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()   # captures what is launched on this stream alone
        with torch.cuda.graph(graph, stream=side):
            o, _ = lr.decay_attn_step(q, k, v, 4, Hk=2, a_log=a, g=g, S=S)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want)
