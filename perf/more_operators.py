"""Cases for measuring the selective scan with heads (one decay per head, B and C shared by groups
of heads), the short causal convolution before it, both as prompts and as single tokens, and the norm
of queries and keys with the position rotation in the same pass.

``run`` computes each operator in plain 32-bit torch, or through the library's public calls where
``own`` is true.  Inputs follow the library's own workload generators: activations ~ N(0, 1), step
sizes log-uniform over 1e-3 .. 1e-1 before noise, decay rates 1 .. 16 spread over the heads.  As in a
layer, the inputs are slices of one projection's output, so their rows lie apart in memory.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def _conv(name, B, L, C, W, io, act="silu", ragged=False, state=False, apart=0):
    """apart: columns of the projection beside x's (0: x is dense)."""
    c = {"op": "conv", "B": B, "L": L, "C": C, "W": W, "io": io, "act": act, "ragged": ragged,
         "state": state, "apart": apart}
    return dict(c, name=name) if name else c


def _conv_step(name, B, C, W, io, act="silu", apart=0):
    c = {"op": "conv_step", "B": B, "C": C, "W": W, "io": io, "act": act, "apart": apart}
    return dict(c, name=name) if name else c


def _heads(name, B, L, H, G, P, N, io, gate=True, skip=True, ragged=False, state=False):
    c = {"op": "heads", "B": B, "L": L, "H": H, "G": G, "P": P, "N": N, "io": io, "gate": gate,
         "skip": skip, "ragged": ragged, "state": state}
    return dict(c, name=name) if name else c


def _heads_step(name, B, H, G, P, N, io, gate=True):
    c = {"op": "heads_step", "B": B, "H": H, "G": G, "P": P, "N": N, "io": io, "gate": gate}
    return dict(c, name=name) if name else c


def _rope(name, B, L, H, Hk, d, rot, io, norm="rms", pairs="halves", start=0):
    c = {"op": "rope", "B": B, "L": L, "H": H, "Hk": Hk, "d": d, "rot": rot, "io": io, "norm": norm,
         "pairs": pairs, "start": start}
    return dict(c, name=name) if name else c


def listed():
    return [
        # the convolution over x, B and C of a batch of prompts (16 heads of 128 and two times 128)
        _conv("conv_b4_l4096", 4, 4096, 2304, 4, "bf16", apart=2064),
        # a ragged batch in fp32, resumed, three taps, an odd width
        _conv("conv_ragged_f32_w3", 8, 1017, 1321, 3, "f32", ragged=True, state=True),
        # decode: one sequence (latency) and a serving batch
        _conv_step("conv_step_b1", 1, 2304, 4, "bf16", apart=2064),
        _conv_step("conv_step_b64", 64, 2304, 4, "bf16", apart=2064),
        # the scan of the same batch of prompts, with skip and gate
        _heads("heads_b4_l4096", 4, 4096, 16, 1, 128, 128, "bf16"),
        # one long prompt: few heads in flight, the sequence itself has to be split
        _heads("heads_b1_l32768", 1, 32768, 16, 1, 128, 128, "bf16", gate=False),
        # a ragged batch resumed from states, 64-wide heads, B and C of two groups
        _heads("heads_ragged_p64", 8, 1017, 32, 2, 64, 64, "bf16", ragged=True, state=True),
        # fp32 activations, a short prompt whose sizes are no powers of two
        _heads("heads_f32_p80", 2, 700, 12, 3, 80, 96, "f32"),
        # decode: a serving batch, and one sequence
        _heads_step("heads_step_b64", 64, 16, 1, 128, 128, "bf16"),
        _heads_step("heads_step_b1", 1, 16, 1, 128, 128, "bf16"),
        # queries and keys of a batch of prompts: 16 heads share 4 key heads
        _rope("norm_rope_b4_l4096", 4, 4096, 16, 4, 128, 128, "bf16"),
        # decode far into a sequence, half of each head rotated, neighbouring pairs
        _rope("norm_rope_decode_b8", 8, 1, 16, 4, 128, 64, "bf16", pairs="neighbours", start=1 << 20),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    io = "bf16" if rng.random() < 0.7 else "f32"
    op = rng.choice(["conv", "conv", "conv_step", "heads", "heads", "heads_step", "rope"])
    if op in ("conv", "conv_step"):
        C = rng.choice([64, 333, 768, 1000, 1321, 2304, 4352])
        W = rng.choice([2, 3, 4, 4, 4])
        act = rng.choice(["silu", "silu", "none"])
        apart = rng.choice([0, 0, 16, 1040, 2064])
        if op == "conv_step":
            return _conv_step(None, _logint(rng, 1, 256), C, W, io, act, apart)
        B = _logint(rng, 1, 8)
        L = _logint(rng, 1, min(16384, (4 * 4096 * 2304 // (2 if io == "f32" else 1)) // (B * C)))
        return _conv(None, B, L, C, W, io, act, rng.random() < 0.3, rng.random() < 0.5, apart)
    if op == "rope":
        d = rng.choice([32, 64, 80, 96, 128, 128, 128, 192, 256])
        Hk = rng.choice([1, 2, 3, 4, 8])
        H = Hk * rng.choice([1, 2, 4])
        rot = rng.choice([d, d, d // 2])
        B = _logint(rng, 1, 8)
        L = _logint(rng, 1, min(16384, (4 * 4096 * 20 * 128 // (2 if io == "f32" else 1)) // (B * (H + Hk) * d)))
        return _rope(None, B, L, H, Hk, d, rot, io, rng.choice(["rms", "rms", "l2", "none"]),
                     rng.choice(["halves", "neighbours"]), rng.choice([0, 0, 5000, 1 << 20]))
    P = rng.choice([32, 64, 64, 72, 80, 128, 128])
    N = rng.choice([16, 32, 64, 64, 96, 128, 128, 128, 256])
    G = rng.choice([1, 1, 1, 2, 3, 8])
    H = G * rng.choice([2, 4, 8])
    if op == "heads_step":
        B = _logint(rng, 1, max(1, min(256, (1 << 24) // (H * P * N))))
        return _heads_step(None, B, H, G, P, N, io, rng.random() < 0.6)
    B = _logint(rng, 1, 8)
    budget = 4 * 4096 * 16 * 256 // (2 if io == "f32" else 1)
    L = _logint(rng, 1, max(1, min(16384, budget // (B * H * (P + N)))))
    return _heads(None, B, L, H, G, P, N, io, rng.random() < 0.6, rng.random() < 0.7,
                  rng.random() < 0.3, rng.random() < 0.5)


# ----------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = _DT[case["io"]]
    c = case

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev) * std

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=g, device=dev) * (hi - lo) + lo

    def lengths():
        return torch.randint(0, c["L"] + 1, (c["B"],), generator=g, device=dev).to(torch.int32)

    if c["op"] in ("conv", "conv_step"):
        n = (c["B"], c["L"]) if c["op"] == "conv" else (c["B"],)
        # the projection puts its other parts before x
        st = {"x": normal(*n, c["apart"] + c["C"]).to(dt)[..., c["apart"]:]}
        st["w"] = uniform(c["C"], c["W"], lo=-1.0, hi=1.0) * c["W"] ** -0.5
        st["bias"] = 0.1 * normal(c["C"])
        st["lens"] = lengths() if c.get("ragged") else None
        keep = c["op"] == "conv_step" or c["state"]
        st["state"] = normal(c["B"], c["W"] - 1, c["C"]).to(dt) if keep else None
        if c["op"] == "conv_step":
            st["state_out"] = torch.empty_like(st["state"])
        return {"case": case, **st}
    if c["op"] == "rope":
        H, Hk, d = c["H"], c["Hk"], c["d"]
        qkv = normal(c["B"], c["L"], (H + 2 * Hk) * d, std=1.5).to(dt)
        pos = c["start"] + torch.randint(0, 100, (c["B"], 1), generator=g, device=dev) * (c["start"] > 0)
        pos = (pos + torch.arange(c["L"], device=dev)).to(torch.int32)
        i = torch.arange(c["rot"] // 2, device=dev, dtype=torch.float64)
        return {"case": case, "q": qkv[..., :H * d], "k": qkv[..., H * d:(H + Hk) * d], "pos": pos.contiguous(),
                "freqs": (10000.0 ** (-2.0 * i / c["rot"])).float(),
                "gamma_q": 1.0 + 0.1 * normal(d), "gamma_k": 1.0 + 0.1 * normal(d)}
    B, H, G, P, N = (c[n] for n in ("B", "H", "G", "P", "N"))
    n = (B, c["L"]) if c["op"] == "heads" else (B,)
    # z and dt from the projection, x, B and C from the convolution
    zdt = normal(*n, H * P + H)
    zdt[..., H * P:] = 0.5 * zdt[..., H * P:]
    zdt, xbc = zdt.to(dt), normal(*n, H * P + 2 * G * N).to(dt)
    st = {"x": xbc[..., :H * P], "Bm": xbc[..., H * P:H * P + G * N], "Cm": xbc[..., H * P + G * N:],
          "dt": zdt[..., H * P:], "z": zdt[..., :H * P] if c["gate"] else None}
    size = torch.exp(uniform(H, lo=math.log(1e-3), hi=math.log(1e-1)))
    st["dt_bias"] = torch.log(torch.expm1(size))                 # softplus of it is the size
    st["A_log"] = torch.log(uniform(H, lo=1.0, hi=16.0))
    st["Dskip"] = 1.0 + 0.1 * normal(H) if c.get("skip", True) else None
    if c["op"] == "heads_step":
        st["S"] = 0.5 * normal(B, H, P, N)
        st["S_out"] = torch.empty_like(st["S"])
        return {"case": case, **st}
    st["S0"] = 0.5 * normal(B, H, P, N) if c["state"] else None
    st["lens"] = lengths() if c["ragged"] else None
    return {"case": case, **st}


# ------------------------------------------------------------ plain forms
def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _plain_conv(s):
    c = s["case"]
    one = c["op"] == "conv_step"
    x = s["x"][:, None] if one else s["x"]
    (B, L, C), W, dt = x.shape, c["W"], x.dtype
    state = x.new_zeros(B, W - 1, C) if s["state"] is None else s["state"]
    xs = torch.cat([state, x], 1)                                # input t at W - 1 + t
    y = s["bias"].expand(B, L, C)
    for j in range(W):
        y = y + s["w"][:, j] * xs[:, j:j + L].float()
    if c["act"] == "silu":
        y = _silu(y)
    if s["lens"] is None:
        new = xs[:, L:]
    else:
        ok = torch.arange(L, device=x.device) < s["lens"][:, None]
        y = torch.where(ok[..., None], y, torch.zeros((), device=x.device))
        at = s["lens"].long()[:, None] + torch.arange(W - 1, device=x.device)
        new = torch.gather(xs, 1, at[..., None].expand(B, W - 1, C))
    y = y.to(dt)
    return {"y": y[:, 0] if one else y, "state": new.contiguous()}


def _delta(s):
    d = s["dt"].float() + s["dt_bias"]
    return torch.where(d > 20.0, d, torch.log1p(torch.exp(d)))


def _split(t, n, H):
    """(B, L, n*d) -> (B, H, L, d) in 32 bits, groups repeated over their heads."""
    B, L, D = t.shape
    t = t.float().reshape(B, L, n, D // n).transpose(1, 2)
    return t if n == H else t.repeat_interleave(H // n, dim=1)


def _segsum(l):
    """sum of l over (s, t] for s <= t along the last axis, -inf above the diagonal."""
    n = l.shape[-1]
    i = torch.arange(n, device=l.device)
    x = l.unsqueeze(-1).expand(*l.shape, n)
    x = torch.where(i[:, None] > i[None, :], x, torch.zeros((), device=l.device))
    x = x.cumsum(-2)
    return torch.where(i[:, None] >= i[None, :], x, torch.full((), -math.inf, device=l.device))


def _plain_heads(s):
    c = s["case"]
    H, G, P, N, dt = c["H"], c["G"], c["P"], c["N"], s["x"].dtype
    B, L, _ = s["x"].shape
    x, Bm, Cm = _split(s["x"], H, H), _split(s["Bm"], G, H), _split(s["Cm"], G, H)
    delta = _delta(s).transpose(1, 2)                            # (B, H, L)
    if s["lens"] is not None:
        ok = (torch.arange(L, device=x.device) < s["lens"][:, None])[:, None, :]
        delta = delta * ok
    l = -torch.exp(s["A_log"])[:, None] * delta
    v = x * delta[..., None]
    C = min(64, L)
    n = (L + C - 1) // C
    pad = n * C - L
    if pad:
        v, Bm, Cm = (torch.cat([t, t.new_zeros(B, H, pad, t.shape[-1])], 2) for t in (v, Bm, Cm))
        l = torch.cat([l, l.new_zeros(B, H, pad)], 2)
    v, Bm, Cm = (t.reshape(B, H, n, C, -1) for t in (v, Bm, Cm))
    l = l.reshape(B, H, n, C)
    seg = _segsum(l)                                             # within a chunk
    y = ((Cm @ Bm.transpose(-1, -2)) * torch.exp(seg)) @ v
    dS = (v * torch.exp(seg[..., -1, :])[..., None]).transpose(-1, -2) @ Bm    # (B, H, n, P, N)
    tot = l.sum(-1)
    # state before chunk c (c = n: the final one): all earlier chunks', decayed
    S0 = torch.zeros(B, H, P, N, device=x.device) if s["S0"] is None else s["S0"]
    src = torch.cat([S0[:, :, None], dS], 2).reshape(B, H, n + 1, P * N)
    S = torch.exp(_segsum(torch.cat([tot.new_zeros(B, H, 1), tot], 2))) @ src
    S = S.reshape(B, H, n + 1, P, N)
    y = y + torch.exp(l.cumsum(-1))[..., None] * (Cm @ S[:, :, :-1].transpose(-1, -2))
    y = y.reshape(B, H, n * C, P)[:, :, :L]
    if s["Dskip"] is not None:
        y = y + s["Dskip"][:, None, None] * x
    y = y.transpose(1, 2).reshape(B, L, H * P)
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    if s["lens"] is not None:
        y = torch.where(ok[:, 0, :, None], y, torch.zeros((), device=x.device))
    return {"y": y.to(dt), "S": S[:, :, -1].contiguous()}


def _plain_heads_step(s):
    c = s["case"]
    H, G, dt = c["H"], c["G"], s["x"].dtype
    B = s["x"].shape[0]
    x, Bm, Cm = (_split(s[n][:, None], h, H)[:, :, 0] for n, h in (("x", H), ("Bm", G), ("Cm", G)))
    delta = _delta(s)
    a = torch.exp(-torch.exp(s["A_log"]) * delta)
    S = a[..., None, None] * s["S"] + (delta[..., None] * x)[..., :, None] * Bm[..., None, :]
    y = (S * Cm[..., None, :]).sum(-1)
    if s["Dskip"] is not None:
        y = y + s["Dskip"][:, None] * x
    y = y.reshape(B, -1)
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return {"y": y.to(dt), "S": S}


def _plain_rope(s):
    c = s["case"]
    d, rot = c["d"], c["rot"]
    angle = s["pos"].double()[..., None] * s["freqs"].double()   # far positions need the bits
    cos, sin = torch.cos(angle).float()[..., None, :], torch.sin(angle).float()[..., None, :]

    def one(x, gamma):
        t = x.float().reshape(*x.shape[:-1], -1, d)
        if c["norm"] == "rms":
            t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * gamma
        elif c["norm"] == "l2":
            t = t / torch.sqrt((t * t).sum(-1, keepdim=True) + 1e-6) * gamma
        if c["pairs"] == "halves":
            a, b = t[..., :rot // 2], t[..., rot // 2:rot]
            t = torch.cat([a * cos - b * sin, b * cos + a * sin, t[..., rot:]], -1)
        else:
            a, b = t[..., 0:rot:2], t[..., 1:rot:2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
            t = torch.cat([r, t[..., rot:]], -1)
        return t.reshape(x.shape).to(x.dtype)

    return {"q": one(s["q"], s["gamma_q"]), "k": one(s["k"], s["gamma_k"])}


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"conv": _plain_conv, "conv_step": _plain_conv, "heads": _plain_heads,
                "heads_step": _plain_heads_step, "rope": _plain_rope}[c["op"]](s)
    from selective_state_space_chunked_gb300 import binding as lr
    if c["op"] == "conv":
        y, new = lr.causal_conv(s["x"], s["w"], bias=s["bias"], state=s["state"], lens=s["lens"], act=c["act"])
        return {"y": y, "state": new}
    if c["op"] == "conv_step":
        y, new = lr.causal_conv_step(s["x"], s["w"], bias=s["bias"], state=s["state"],
                                     state_out=s["state_out"], act=c["act"])
        return {"y": y, "state": new}
    if c["op"] == "heads":
        y, S = lr.selective_heads(s["x"], s["dt"], s["Bm"], s["Cm"], s["A_log"], c["H"], G=c["G"], z=s["z"],
                                  Dskip=s["Dskip"], dt_bias=s["dt_bias"], S0=s["S0"], lens=s["lens"])
        return {"y": y, "S": S}
    if c["op"] == "heads_step":
        y, S = lr.selective_heads_step(s["x"], s["dt"], s["Bm"], s["Cm"], s["A_log"], c["H"], G=c["G"],
                                       z=s["z"], Dskip=s["Dskip"], dt_bias=s["dt_bias"], S=s["S"],
                                       S_out=s["S_out"])
        return {"y": y, "S": S}
    with_norm = c["norm"] != "none"
    q, k = lr.head_norm_rope(s["q"], s["k"], c["H"], Hk=c["Hk"], norm=c["norm"],
                             gamma_q=s["gamma_q"] if with_norm else None,
                             gamma_k=s["gamma_k"] if with_norm else None, freqs=s["freqs"], pos=s["pos"],
                             pairs=c["pairs"], eps=1e-6)
    return {"q": q, "k": k}


# -------------------------------------------------------------- work, exact
def work(case):
    c = case
    es = 2 if c["io"] == "bf16" else 4
    if c["op"] in ("conv", "conv_step"):
        T, keep = c["B"] * c.get("L", 1), c["B"] * (c["W"] - 1) * c["C"]
        part = 0.5 if c.get("ragged") else 1.0                   # of the inputs; outputs are whole
        states = 2 if c["op"] == "conv_step" or c["state"] else 1
        return {"bytes": int(es * T * c["C"] * (1.0 + part)) + es * keep * states + 4 * c["C"] * (c["W"] + 1),
                "flops": int(part * T * c["C"] * (2 * c["W"] + (4 if c["act"] == "silu" else 0)))}
    if c["op"] == "rope":
        n = c["B"] * c["L"] * (c["H"] + c["Hk"]) * c["d"]
        return {"bytes": 2 * es * n + 4 * c["B"] * c["L"] + 8 * c["d"] + 2 * c["rot"], "flops": 7 * n}
    B, H, G, P, N = (c[n] for n in ("B", "H", "G", "P", "N"))
    tok = es * (H * P * (2 if c["gate"] else 1) + 2 * G * N + H)  # read
    head, state = 4 * H * 3, 4 * B * H * P * N
    if c["op"] == "heads_step":
        return {"bytes": B * (tok + es * H * P) + head + 2 * state, "flops": 6 * B * H * P * N}
    T = B * c["L"]
    part = 0.5 if c["ragged"] else 1.0
    return {"bytes": int(T * (part * tok + es * H * P)) + head + state * (2 if c["state"] else 1),
            "flops": int(part * 4 * T * H * P * N)}


def _np(t):
    return t.double().cpu().numpy()


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] in ("conv", "conv_step"):
        x, w, b = _np(s["x"]), _np(s["w"]), _np(s["bias"])
        if c["op"] == "conv_step":
            x = x[:, None]
        B, L, C = x.shape
        W = c["W"]
        old = np.zeros((B, W - 1, C)) if s["state"] is None else _np(s["state"])
        y, new = np.zeros((B, L, C)), np.zeros((B, W - 1, C))
        for r in range(B):
            n = L if s["lens"] is None else int(s["lens"][r])
            v = np.concatenate([old[r], x[r, :n]])
            acc = np.tile(b, (n, 1))
            for j in range(W):
                acc += w[:, j] * v[j:j + n]
            y[r, :n] = acc / (1.0 + np.exp(-acc)) if c["act"] == "silu" else acc
            new[r] = v[len(v) - (W - 1):]
        return {"y": y[:, 0] if c["op"] == "conv_step" else y, "state": new}
    if c["op"] == "rope":
        d, rot = c["d"], c["rot"]
        turn = np.exp(1j * (_np(s["pos"])[..., None] * _np(s["freqs"])))[..., None, :]
        out = {}
        for n, gamma in (("q", "gamma_q"), ("k", "gamma_k")):
            x = _np(s[n])
            shape = x.shape
            x = x.reshape(*shape[:-1], -1, d).copy()
            if c["norm"] != "none":
                q = (x * x).sum(-1, keepdims=True)
                x = x / np.sqrt((q / d if c["norm"] == "rms" else q) + 1e-6) * _np(s[gamma])
            lo = slice(0, rot // 2) if c["pairs"] == "halves" else slice(0, rot, 2)
            hi = slice(rot // 2, rot) if c["pairs"] == "halves" else slice(1, rot, 2)
            p = (x[..., lo] + 1j * x[..., hi]) * turn
            x[..., lo], x[..., hi] = p.real, p.imag
            out[n] = x.reshape(shape)
        return out
    # the recurrence itself, a token at a time
    f64 = torch.float64
    B, H, G, P, N = (c[n] for n in ("B", "H", "G", "P", "N"))
    one = c["op"] == "heads_step"
    L = 1 if one else c["L"]
    idx = torch.arange(H, device="cuda") // (H // G)
    x = s["x"].to(f64).reshape(B, L, H, P)
    Bm = s["Bm"].to(f64).reshape(B, L, G, N)
    Cm = s["Cm"].to(f64).reshape(B, L, G, N)
    delta = torch.logaddexp(s["dt"].to(f64).reshape(B, L, H) + s["dt_bias"].to(f64),
                            torch.zeros((), dtype=f64, device="cuda"))
    a = torch.exp(-torch.exp(s["A_log"].to(f64)) * delta)
    lens = [L] * B if one or s["lens"] is None else s["lens"].tolist()
    S = s["S"] if one else s["S0"]
    S = torch.zeros(B, H, P, N, dtype=f64, device="cuda") if S is None else S.to(f64).clone()
    y = torch.zeros(B, L, H, P, dtype=f64, device="cuda")
    order = sorted(range(B), key=lambda b: -lens[b])             # rows still running come first
    perm = torch.tensor(order, device="cuda")
    x, Bm, Cm, delta, a, S = (t[perm] for t in (x, Bm, Cm, delta, a, S))
    for t in range(L):
        n = sum(v > t for v in lens)
        if n == 0:
            break
        S[:n] *= a[:n, t, :, None, None]
        S[:n].addcmul_((delta[:n, t, :, None] * x[:n, t])[..., None], Bm[:n, t][:, idx][:, :, None, :])
        y[:n, t] = torch.matmul(S[:n], Cm[:n, t][:, idx][..., None])[..., 0]
        if s["Dskip"] is not None:
            y[:n, t] += s["Dskip"].to(f64)[:, None] * x[:n, t]
    back = torch.argsort(perm)
    y, S = y[back].reshape(B, L, H * P), S[back]
    if s["z"] is not None:
        z = s["z"].to(f64).reshape(B, L, H * P)
        y = y * (z / (1.0 + torch.exp(-z)))
    return {"y": y[:, 0] if one else y, "S": S}
