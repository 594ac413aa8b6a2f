"""The torch helpers of the short convolution, of the selective scan with heads and of the
norm with rotation: their short path gives the helper's own results and declines what is
not already in the kernels' form; calls that follow one another; a failed launch; and the
operators together, as a layer runs them, against the float64 oracle."""
import pytest
import torch

import oracle
from conftest import rel_err
from selective_state_space_chunked_gb300 import workloads as wl
from test_decay_attn_gpu import cuda, lr  # noqa: F401

pytestmark = pytest.mark.gpu
NAMES = ("causal_conv", "causal_conv_step", "selective_heads", "selective_heads_step", "head_norm_rope")


def inputs(io, L=70, B=3, H=4, G=2, P=32, N=16, apart=0):
    """A layer's tensors: slices of one projection's output and of one convolution's."""
    p = cuda(wl.selective_heads_inputs(B, L, H, G, P, N, 5, io=io, with_S0=True))
    xbc = torch.cat([p["x"], p["Bm"], p["Cm"]], -1)
    zdt = torch.cat([p["z"], p["dt"], p["dt"].new_zeros(B, L, apart)], -1)
    C = xbc.shape[-1]
    g = torch.Generator().manual_seed(1)
    return dict(xbc=xbc, x=xbc[..., :H * P], Bm=xbc[..., H * P:H * P + G * N], Cm=xbc[..., H * P + G * N:],
                z=zdt[..., :H * P], dt=zdt[..., H * P:H * P + H], A=p["A_log"], skip=p["Dskip"], bias=p["dt_bias"], S=p["S0"],
                w=(torch.rand(C, 4, generator=g) - 0.5).cuda(), b=torch.randn(C, generator=g).cuda(),
                cs=torch.randn(B, 3, C, generator=g).to(xbc.dtype).cuda(), H=H, G=G,
                lens=torch.tensor([L, 0, 33, 5][:B], dtype=torch.int32).cuda(), gamma=torch.randn(N, generator=g).cuda(),
                freqs=(0.1 ** torch.arange(N // 2)).cuda(),
                pos=torch.arange(L, dtype=torch.int32).expand(B, L).contiguous().cuda())


def calls(lr, d):  # noqa: F811
    """One call of each helper, with and without its optional arguments."""
    one = lambda n: d[n][:, 0]  # noqa: E731
    S, cs = d["S"].clone(), d["cs"].clone()
    kw = dict(G=d["G"], Dskip=d["skip"], dt_bias=d["bias"])
    out = [*lr.causal_conv(d["xbc"], d["w"], bias=d["b"], state=d["cs"], lens=d["lens"]),
           *lr.causal_conv(d["x"], d["w"][:d["x"].shape[-1]], act="none"),
           *lr.causal_conv_step(one("xbc"), d["w"], bias=d["b"], state=cs, state_out=cs),
           *lr.causal_conv_step(one("x"), d["w"][:d["x"].shape[-1]]),
           *lr.selective_heads(d["x"], d["dt"], d["Bm"], d["Cm"], d["A"], d["H"], z=d["z"], S0=d["S"], lens=d["lens"], **kw),
           *lr.selective_heads(d["x"], d["dt"], d["Bm"], d["Cm"], d["A"], d["H"], G=d["G"]),
           *lr.selective_heads_step(one("x"), one("dt"), one("Bm"), one("Cm"), d["A"], d["H"], z=one("z"), S=S, S_out=S,
                                    **kw),
           *lr.selective_heads_step(one("x"), one("dt"), one("Bm"), one("Cm"), d["A"], d["H"], G=d["G"]),
           *lr.head_norm_rope(d["Cm"], d["Bm"], d["G"], gamma_q=d["gamma"], freqs=d["freqs"], pos=d["pos"]),
           lr.head_norm_rope(d["x"], None, d["H"], norm="l2")[0]]
    lr.check_status()
    return out


# z's rows leave 16-byte boundaries in bf16 where nothing stands beside them: the prompt's z
# is then copied, by the short path too
@pytest.mark.parametrize("io,apart,declined", [("bf16", 0, []), ("bf16", 4, []), ("f32", 0, [])])
def test_the_short_path_gives_the_helpers_results(lr, io, apart, declined, monkeypatch):  # noqa: F811
    d = inputs(io, apart=apart)
    taken = []
    for name in NAMES:
        f = getattr(lr._lrtorch, name)
        monkeypatch.setattr(lr._lrtorch, name, lambda *a, f=f: taken.append(f(*a)) or taken[-1])
    short = calls(lr, d)
    assert len(taken) == 10 and [i for i, r in enumerate(taken) if type(r) is not tuple] == declined
    for name in NAMES:
        monkeypatch.setattr(lr._lrtorch, name, lambda *a: None)
    long = calls(lr, d)
    assert len(short) == len(long) == 19
    for a, b in zip(short, long):
        assert torch.equal(a, b)


def test_what_is_declined_is_converted_or_refused(lr):  # noqa: F811
    d = inputs("f32")
    good = (d["xbc"], d["w"], d["b"], d["cs"], d["lens"], 1)
    want = lr._lrtorch.causal_conv(*good)
    assert want is not None
    for i, other in [(0, d["xbc"].cpu()), (0, d["xbc"].half()), (0, d["xbc"][:, :0]), (0, None), (1, d["w"].double()),
                     (1, d["w"].t()), (1, d["w"][:, :1]), (2, d["b"][1:]), (3, d["cs"].bfloat16()), (3, d["cs"][:, :2]),
                     (4, d["lens"].long()), (5, None)]:
        args = list(good)
        args[i] = other
        assert lr._lrtorch.causal_conv(*args) is None, i
    got = lr.causal_conv(d["xbc"], d["w"].double(), bias=d["b"].double(), state=d["cs"], lens=d["lens"].long())
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    off = torch.empty(d["xbc"].numel() + 1, device="cuda")[1:].view_as(d["xbc"]).copy_(d["xbc"])   # off 16 bytes
    assert lr._lrtorch.causal_conv(off, *good[1:]) is None
    assert torch.equal(lr.causal_conv(off, d["w"], bias=d["b"], state=d["cs"], lens=d["lens"])[0], want[0])
    q = (d["x"], d["dt"], d["Bm"], d["Cm"], d["A"], 4, 2, d["z"], d["skip"], d["bias"], d["S"], d["lens"], True)
    assert lr._lrtorch.selective_heads(*q) is not None
    for i, other in [(0, d["x"].bfloat16()), (1, d["dt"][..., :3]), (2, d["Bm"][:, ::2]), (3, d["Cm"].cpu()), (5, 3), (6, 3),
                     (7, d["z"][..., :-1]), (10, d["S"].transpose(2, 3)), (11, d["lens"][:2])]:
        args = list(q)
        args[i] = other
        assert lr._lrtorch.selective_heads(*args) is None, i
    with pytest.raises(ValueError):
        lr.selective_heads(d["x"], d["dt"], d["Bm"], d["Cm"], d["A"], 4, G=2, lens=d["lens"][:2])
    r = (d["Cm"], d["Bm"], 2, None, 1, d["gamma"], None, d["freqs"], d["pos"], 0, 1e-6)
    assert lr._lrtorch.head_norm_rope(*r) is not None
    for i, other in [(0, d["Cm"].double()), (1, d["Bm"][..., :-1]), (2, 3), (3, 4), (5, d["gamma"][1:]),
                     (7, torch.ones(9, device="cuda")), (8, None), (8, d["pos"].long()), (4, None)]:
        args = list(r)
        args[i] = other
        assert lr._lrtorch.head_norm_rope(*args) is None, i


def test_a_failed_launch_is_raised_not_repeated(lr, monkeypatch):  # noqa: F811
    d = inputs("f32")
    for name in NAMES:
        monkeypatch.setattr(lr._lrtorch, name, lambda *a: lr.LR_ERR_CUDA)
    S, cs = d["S"].clone(), d["cs"].clone()
    one = lambda n: d[n][:, 0]  # noqa: E731
    for f in (lambda: lr.causal_conv(d["xbc"], d["w"]),
              lambda: lr.causal_conv_step(one("xbc"), d["w"], state=cs, state_out=cs),
              lambda: lr.selective_heads(d["x"], d["dt"], d["Bm"], d["Cm"], d["A"], 4, G=2),
              lambda: lr.selective_heads_step(one("x"), one("dt"), one("Bm"), one("Cm"), d["A"], 4, G=2, S=S, S_out=S),
              lambda: lr.head_norm_rope(d["Cm"], d["Bm"], 2)):
        with pytest.raises(lr.LrError):
            f()
    assert torch.equal(S, d["S"]) and torch.equal(cs, d["cs"])


# fp32: sums of up to a few hundred terms in another order, 300 * 2^-24 = 2e-5, through a
# norm: 1e-4.  bf16: each operator rounds its output by 2^-8 of it and the next carries
# that on: four of them in a row (convolution, norm, scan, norm), a norm raising the error
# of a value that is a third of its group's size to three times that: 5e-2.
@pytest.mark.parametrize("io,tol,tol_s", [("f32", 1e-4, 1e-4), ("bf16", 5e-2, 3e-2)])
@pytest.mark.parametrize("L,n", [(1, 0), (40, 3), (200, 60)])
def test_together_as_a_layer(lr, io, tol, tol_s, L, n):  # noqa: F811
    """Convolution, norm and rotation of B and C, scan with gate, norm: a prompt of ragged
    rows, then tokens in place of the states, each call starting while the one before it
    drains, against the oracle's operators on whole rows."""
    B, H, G, P, N = 3, 4, 2, 64, 32
    d = inputs(io, L + n, B, H, G, P, N)
    lens = [L, max(L - 7, 0), 0]
    HP, GN = H * P, G * N
    kw = dict(G=G, Dskip=d["skip"], dt_bias=d["bias"])

    def front(y, pos):
        # the scan's B and C; x stays where the convolution put it
        Cm, Bm = lr.head_norm_rope(y[..., HP + GN:], y[..., HP:HP + GN], G, gamma_q=d["gamma"], gamma_k=d["gamma"],
                                   freqs=d["freqs"], pos=pos)
        return y[..., :HP], Bm, Cm

    length = torch.tensor(lens, dtype=torch.int32).cuda()
    y, cs = lr.causal_conv(d["xbc"][:, :L], d["w"], bias=d["b"], lens=length)
    x, Bm, Cm = front(y, d["pos"][:, :L].contiguous())
    y, S = lr.selective_heads(x, d["dt"][:, :L], Bm, Cm, d["A"], H, z=d["z"][:, :L], lens=length, **kw)
    outs = [lr.group_norm_act(y, H)]
    for t in range(L, L + n):   # row b's token follows its own length
        y, _ = lr.causal_conv_step(d["xbc"][:, t], d["w"], bias=d["b"], state=cs, state_out=cs)
        x, Bm, Cm = front(y, length + (t - L))
        y, _ = lr.selective_heads_step(x, d["dt"][:, t], Bm, Cm, d["A"], H, z=d["z"][:, t], S=S, S_out=S, **kw)
        outs.append(lr.group_norm_act(y, H)[:, None])
    got = torch.cat(outs, 1)
    lr.check_status()
    c = {k: v.float().cpu() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in d.items()}
    for b, m in enumerate(lens):
        rows = torch.cat([torch.arange(m), torch.arange(L, L + n)])
        if len(rows) == 0:
            assert not got[b].any() and not S[b].any() and not cs[b].any()
            continue
        yr, csr = oracle.causal_conv(c["xbc"][b:b + 1, rows], c["w"], c["b"])
        pos = torch.arange(len(rows))[None]
        Cr = oracle.head_norm_rope(yr[..., HP + GN:], G, "rms", c["gamma"], c["freqs"], pos)
        Br = oracle.head_norm_rope(yr[..., HP:HP + GN], G, "rms", c["gamma"], c["freqs"], pos)
        yr, Sr = oracle.selective_heads(yr[..., :HP], c["dt"][b:b + 1, rows], Br, Cr, c["A"], H, G=G,
                                        z=c["z"][b:b + 1, rows], Dskip=c["skip"], dt_bias=c["bias"])
        ref = oracle.group_norm_act(yr[0], H)
        assert rel_err(got[b, rows].float().cpu(), ref) <= tol
        assert rel_err(S[b].cpu(), Sr[0]) <= tol_s and rel_err(cs[b].float().cpu(), csr[0]) == 0.0
        assert not got[b, m:L].any()


def layer(lr, d, L):  # noqa: F811
    """The operators of a prompt in a row."""
    HP, GN, G, H = d["x"].shape[-1], d["Bm"].shape[-1], d["G"], d["H"]
    y, cs = lr.causal_conv(d["xbc"], d["w"], bias=d["b"])
    Cm, Bm = lr.head_norm_rope(y[..., HP + GN:], y[..., HP:HP + GN], G, gamma_q=d["gamma"], freqs=d["freqs"], pos=d["pos"])
    y, S = lr.selective_heads(y[..., :HP], d["dt"], Bm, Cm, d["A"], H, G=G, z=d["z"], Dskip=d["skip"], dt_bias=d["bias"])
    return lr.group_norm_act(y, H), cs, S


@pytest.mark.parametrize("L", [30, 300, 3000])
def test_a_layer_captured_and_replayed_on_new_inputs(lr, L):  # noqa: F811
    d = inputs("bf16", L=L, B=1, P=64, N=64)
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer(lr, d, L)
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            got = layer(lr, d, L)
    for k in range(3):
        gen = torch.Generator(device="cuda").manual_seed(k)
        d["xbc"].normal_(generator=gen)
        d["z"].normal_(generator=gen)
        torch.cuda.synchronize()
        want = [t.clone() for t in layer(lr, d, L)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_streams_at_once(lr):  # noqa: F811
    ds = [inputs("bf16", L=900, B=2 + i, P=64, N=64) for i in range(2)]
    for d in ds:
        d["xbc"].normal_(generator=torch.Generator(device="cuda").manual_seed(d["xbc"].shape[0]))
    want = [layer(lr, d, 900) for d in ds]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in ds], [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(layer(lr, ds[i], 900))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            for a, b in zip(r, want[i]):
                assert torch.equal(a, b)
