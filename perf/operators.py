"""Cases for measuring the decayed linear attention (prompt and single-token forms) and the group
norm with activation that follows its readout.

``run`` computes each operator in plain 32-bit torch, or through the library's public calls where
``own`` is true.  Inputs follow the library's own workload generators: q, k, v ~ N(0, 1/128)-like,
gates from sigmoid(f) with f ~ N(2, 1) and above, per-head decays 1 - 2^-(5 .. 12).
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def _attn(name, B, L, H, Hk, dk, dv, io, decay, ragged=False, state=False):
    c = {"op": "decay_attn", "B": B, "L": L, "H": H, "Hk": Hk, "dk": dk, "dv": dv, "io": io,
         "decay": decay, "ragged": ragged, "state": state}
    return dict(c, name=name) if name else c


def _step(name, B, H, Hk, dk, dv, io, decay):
    c = {"op": "decay_attn_step", "B": B, "H": H, "Hk": Hk, "dk": dk, "dv": dv, "io": io,
         "decay": decay}
    return dict(c, name=name) if name else c


def _norm(name, N, C, G, io, act, gate, affine):
    c = {"op": "group_norm_act", "N": N, "C": C, "G": G, "io": io, "act": act, "gate": gate,
         "affine": affine}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a batch of prompts at the sizes of the library's HGRN2 workload
        _attn("prompt_b4_l4096", 4, 4096, 16, 16, 128, 128, "bf16", "token"),
        # one long prompt: few heads in flight, the sequence itself has to be split
        _attn("prompt_b1_l32768", 1, 32768, 16, 16, 128, 128, "bf16", "head"),
        # a ragged batch resumed from states, 64-wide heads, two value heads per key head
        _attn("prompt_ragged_d64", 8, 1017, 32, 16, 64, 64, "bf16", "both", True, True),
        # a short chat turn on a warm state: latency
        _attn("prompt_b1_l77", 1, 77, 16, 16, 128, 128, "bf16", "token", False, True),
        # fp32 activations
        _attn("prompt_f32_b2_l2048", 2, 2048, 16, 16, 128, 128, "f32", "token"),
        # head dims off the powers of two, values wider than keys
        _attn("prompt_dk96_dv192", 2, 1500, 12, 12, 96, 192, "bf16", "token", False, True),
        # decode: one sequence, and a serving batch; fp32 with 64-wide keys and odd batch
        _step("step_b1", 1, 16, 16, 128, 128, "bf16", "token"),
        _step("step_b64", 64, 16, 16, 128, 128, "bf16", "token"),
        _step("step_f32_b17_dk64", 17, 24, 8, 64, 128, "f32", "head"),
        # the gated norm on the prompt's readout, on a decode batch's, and with plain silu in fp32
        _norm("norm_gate_b4_l4096", 16384, 2048, 16, "bf16", "none", True, True),
        _norm("norm_gate_decode_b8", 8, 2048, 16, "bf16", "none", True, True),
        _norm("norm_silu_f32_d80", 3001, 1920, 24, "f32", "silu", False, True),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    io = "bf16" if rng.random() < 0.7 else "f32"
    kind = rng.choice(["decay_attn", "decay_attn", "decay_attn_step", "group_norm_act"])
    if kind == "group_norm_act":
        d = rng.choice([32, 48, 64, 80, 96, 100, 128, 128, 192, 256, 500, 1024])
        G = rng.choice([1, 2, 3, 8, 16, 24, 32])
        N = _logint(rng, 1, max(1, min(40000, (1 << 25) // (d * G))))
        return _norm(None, N, d * G, G, io, rng.choice(["none", "silu"]), rng.random() < 0.6,
                     rng.random() < 0.8)
    dk = rng.choice([32, 48, 64, 64, 80, 96, 128, 128, 128, 192, 256])
    dv = rng.choice([32, 64, 64, 72, 96, 128, 128, 128, 192, 256])
    Hk = rng.choice([1, 2, 3, 4, 8, 12, 16])
    H = Hk * rng.choice([1, 1, 1, 2, 4])
    decay = rng.choice(["token", "token", "head", "both"])
    if kind == "decay_attn_step":
        B = _logint(rng, 1, max(1, min(256, (1 << 24) // (H * dk * dv))))
        return _step(None, B, H, Hk, dk, dv, io, decay)
    B = _logint(rng, 1, 8)
    budget = 4 * 4096 * 16 * 256 // (2 if io == "f32" else 1)
    L = _logint(rng, 1, max(1, min(16384, budget // (B * H * (dk + dv)))))
    return _attn(None, B, L, H, Hk, dk, dv, io, decay, rng.random() < 0.3, rng.random() < 0.5)


# ----------------------------------------------------------------- inputs
def _decays(case, n, g, dev):
    """Per-head log decays (H) fp32 and per-token ones (*n, H) in the I/O type, or None."""
    H = case["H"]
    a_log = tok = None
    if case["decay"] in ("head", "both"):
        a = 1.0 - 2.0 ** -(5.0 + 7.0 * torch.arange(H, device=dev) / max(H, 1))
        a_log = torch.log(a).float()
    if case["decay"] in ("token", "both"):
        f = 3.0 + torch.randn(*n, H, generator=g, device=dev)
        tok = torch.log(torch.sigmoid(f)).to(_DT[case["io"]])
    return a_log, tok


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = _DT[case["io"]]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std)

    if case["op"] == "group_norm_act":
        N, C = case["N"], case["C"]
        st = {"x": (normal(N, C, std=1.5) + 0.25).to(dt)}
        st["z"] = normal(N, C).to(dt) if case["gate"] else None
        st["gamma"] = 1.0 + 0.1 * normal(C) if case["affine"] else None
        st["beta"] = 0.1 * normal(C) if case["affine"] else None
        return {"case": case, **st}
    B, H, Hk, dk, dv = (case[n] for n in ("B", "H", "Hk", "dk", "dv"))
    n = (B, case["L"]) if case["op"] == "decay_attn" else (B,)
    st = {"q": normal(*n, Hk * dk, std=dk ** -0.5).to(dt), "k": normal(*n, Hk * dk, std=dk ** -0.5).to(dt),
          "v": normal(*n, H * dv, std=dv ** -0.5).to(dt), "scale": dk ** -0.5}
    st["a_log"], st["g"] = _decays(case, n, g, dev)
    if case["op"] == "decay_attn_step":
        st["S"] = 0.1 * normal(B, H, dv, dk)
        st["S_out"] = torch.empty_like(st["S"])
        return {"case": case, **st}
    st["S0"] = 0.1 * normal(B, H, dv, dk) if case["state"] else None
    st["lens"] = None
    if case["ragged"]:
        st["lens"] = torch.randint(0, case["L"] + 1, (B,), generator=g, device=dev).to(torch.int32)
    return {"case": case, **st}


# ------------------------------------------------------------ plain forms
def _heads(t, n, H):
    """(B, L, H*d) -> (B, n heads, L, d) in 32 bits, key heads repeated over their value heads."""
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


def _log_decay(s, shape, H):
    l = torch.zeros(*shape, H, device=s["q"].device)
    if s["a_log"] is not None:
        l = l + s["a_log"]
    if s["g"] is not None:
        l = l + s["g"].float()
    return l


def _plain_attn(s):
    c = s["case"]
    H, Hk, dt = c["H"], c["Hk"], s["q"].dtype
    B, L, _ = s["q"].shape
    q, k, v = _heads(s["q"], Hk, H), _heads(s["k"], Hk, H), _heads(s["v"], H, H)
    dk, dv = q.shape[-1], v.shape[-1]
    l = _log_decay(s, (B, L), H).transpose(1, 2)                 # (B, H, L)
    ok = None
    if s["lens"] is not None:
        ok = (torch.arange(L, device=q.device) < s["lens"][:, None])[:, None, :]
        l, k = l * ok, k * ok[..., None]
    C = min(64, L)
    n = (L + C - 1) // C
    pad = n * C - L
    if pad:
        q, k, v = (torch.cat([t, t.new_zeros(B, H, pad, t.shape[-1])], 2) for t in (q, k, v))
        l = torch.cat([l, l.new_zeros(B, H, pad)], 2)
    q, k, v = (t.reshape(B, H, n, C, -1) for t in (q, k, v))
    l = l.reshape(B, H, n, C)
    seg = _segsum(l)                                             # within a chunk
    tot = l.sum(-1)
    o = ((q @ k.transpose(-1, -2)) * torch.exp(seg)) @ v
    dS = (v * torch.exp(seg[..., -1, :])[..., None]).transpose(-1, -2) @ k     # (B, H, n, dv, dk)
    # state before chunk c (c = n: the final one): all earlier chunks', decayed
    S0 = torch.zeros(B, H, dv, dk, device=q.device) if s["S0"] is None else s["S0"]
    src = torch.cat([S0[:, :, None], dS], 2).reshape(B, H, n + 1, dv * dk)
    W = torch.exp(_segsum(torch.cat([tot.new_zeros(B, H, 1), tot], 2)))        # (B, H, n+1, n+1)
    S = (W @ src).reshape(B, H, n + 1, dv, dk)
    o = o + torch.exp(l.cumsum(-1))[..., None] * (q @ S[:, :, :-1].transpose(-1, -2))
    o = s["scale"] * o.reshape(B, H, n * C, dv)[:, :, :L]
    if ok is not None:
        o = o * ok[..., None]
    return {"o": o.transpose(1, 2).reshape(B, L, H * dv).to(dt), "S": S[:, :, -1].contiguous()}


def _plain_step(s):
    c = s["case"]
    H, Hk, dt = c["H"], c["Hk"], s["q"].dtype
    q, k, v = (_heads(s[n][:, None], h, H)[:, :, 0] for n, h in (("q", Hk), ("k", Hk), ("v", H)))
    a = torch.exp(_log_decay(s, (q.shape[0],), H))
    S = a[..., None, None] * s["S"] + v[..., :, None] * k[..., None, :]
    o = s["scale"] * (S * q[..., None, :]).sum(-1)
    return {"o": o.reshape(q.shape[0], -1).to(dt), "S": S}


def _plain_norm(s):
    c = s["case"]
    x = s["x"].float().reshape(c["N"], c["G"], -1)
    x = x - x.mean(-1, keepdim=True)
    y = (x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5)).reshape(c["N"], c["C"])
    if s["gamma"] is not None:
        y = y * s["gamma"] + s["beta"]
    if c["act"] == "silu":
        y = y / (1.0 + torch.exp(-y))
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z / (1.0 + torch.exp(-z)))
    return {"y": y.to(s["x"].dtype)}


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"decay_attn": _plain_attn, "decay_attn_step": _plain_step,
                "group_norm_act": _plain_norm}[c["op"]](s)
    from selective_state_space_chunked_gb300 import binding as lr
    if c["op"] == "decay_attn":
        o, S = lr.decay_attn(s["q"], s["k"], s["v"], c["H"], Hk=c["Hk"], a_log=s["a_log"], g=s["g"],
                             S0=s["S0"], lens=s["lens"], scale=s["scale"])
        return {"o": o, "S": S}
    if c["op"] == "decay_attn_step":
        o, S = lr.decay_attn_step(s["q"], s["k"], s["v"], c["H"], Hk=c["Hk"], a_log=s["a_log"],
                                  g=s["g"], S=s["S"], S_out=s["S_out"], scale=s["scale"])
        return {"o": o, "S": S}
    return {"y": lr.group_norm_act(s["x"], c["G"], gamma=s["gamma"], beta=s["beta"], z=s["z"],
                                   act=c["act"], eps=1e-5)}


# -------------------------------------------------------------- work, exact
def work(case):
    es = 2 if case["io"] == "bf16" else 4
    if case["op"] == "group_norm_act":
        n = case["N"] * case["C"]
        return {"bytes": es * n * (3 if case["gate"] else 2) + 8 * case["C"] * case["affine"],
                "flops": 8 * n}
    B, H, Hk, dk, dv = (case[n] for n in ("B", "H", "Hk", "dk", "dv"))
    tok = es * (2 * Hk * dk + 2 * H * dv + H * (case["decay"] != "head"))
    head = 4 * H * (case["decay"] != "token")
    state = 4 * B * H * dk * dv
    if case["op"] == "decay_attn_step":
        return {"bytes": B * tok + head + 2 * state, "flops": 5 * B * H * dk * dv}
    T = B * case["L"]
    if case["ragged"]:   # lengths are uniform over 0 .. L: half of the inputs, all of the outputs
        tok = 0.5 * tok + 0.5 * es * H * dv
    return {"bytes": int(T * tok) + head + state * (2 if case["state"] else 1),
            "flops": (0.5 if case["ragged"] else 1.0) * 4 * T * H * dk * dv}


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "group_norm_act":
        x = s["x"].double().cpu().numpy().reshape(case["N"], case["G"], -1)
        y = ((x - x.mean(-1, keepdims=True)) / np.sqrt(x.var(-1, keepdims=True) + 1e-5))
        y = y.reshape(case["N"], case["C"])
        if case["affine"]:
            y = y * s["gamma"].double().cpu().numpy() + s["beta"].double().cpu().numpy()
        if case["act"] == "silu":
            y = y / (1.0 + np.exp(-y))
        if case["gate"]:
            z = s["z"].double().cpu().numpy()
            y = y * z / (1.0 + np.exp(-z))
        return {"y": y}
    # the recurrence itself, a token at a time
    B, H, Hk, dk, dv = (case[n] for n in ("B", "H", "Hk", "dk", "dv"))
    one = case["op"] == "decay_attn_step"
    L = 1 if one else case["L"]
    idx = torch.arange(H, device="cuda") // (H // Hk)
    q = s["q"].to(f64).reshape(B, L, Hk, dk)
    k = s["k"].to(f64).reshape(B, L, Hk, dk)
    v = s["v"].to(f64).reshape(B, L, H, dv)
    a = torch.ones(B, L, H, dtype=f64, device="cuda")
    if s["a_log"] is not None:
        a = a * torch.exp(s["a_log"].to(f64))
    if s["g"] is not None:
        a = a * torch.exp(s["g"].to(f64).reshape(B, L, H))
    lens = [L] * B if one or s["lens"] is None else s["lens"].tolist()
    S = s["S"] if one else s["S0"]
    S = torch.zeros(B, H, dv, dk, dtype=f64, device="cuda") if S is None else S.to(f64).clone()
    o = torch.zeros(B, L, H, dv, dtype=f64, device="cuda")
    order = sorted(range(B), key=lambda b: -lens[b])     # rows still running come first
    perm = torch.tensor(order, device="cuda")
    q, k, v, a, S = q[perm], k[perm], v[perm], a[perm], S[perm]
    for t in range(L):
        n = sum(x > t for x in lens)
        if n == 0:
            break
        S[:n] *= a[:n, t, :, None, None]
        S[:n].addcmul_(v[:n, t, :, :, None], k[:n, t][:, idx][:, :, None, :])
        o[:n, t] = torch.matmul(S[:n], q[:n, t][:, idx][..., None])[..., 0]
    back = torch.argsort(perm)
    o, S = (s["scale"] * o)[back].reshape(B, L, H * dv), S[back]
    return {"o": o[:, 0] if one else o, "S": S}
