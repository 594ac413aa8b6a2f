"""A selective state-space layer with heads for serving: a prompt in one call, then one
token per call from the two states that the prompt left.

    python examples/selective_layer.py [--batch 4] [--prompt 1024] [--tokens 32]

One projection gives the gate z, the channels x, B and C, and a step size per head.  x, B
and C go through the short causal convolution, B and C are normalised and rotated by the
position, and the scan runs over them:

    z, xbc, dt = u W_in
    x, B, C    = causal_conv(xbc)              (prompt; token: causal_conv_step)
    C, B       = head_norm_rope(C, B)
    y          = selective_heads(x, dt, B, C)  (token: selective_heads_step), gated by silu(z)
    out        = group_norm(y) W_out

The kernels read the slices of the projection's and the convolution's outputs where they
stand.  The script prints the times of both phases and how far the tokens' outputs are from
those of one prompt call over the whole sequence.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from selective_state_space_chunked_gb300 import binding as lr  # noqa: E402


class SelectiveLayer:
    """H heads of P channels with N states each; B and C of G groups of heads."""

    def __init__(self, width, H, G, P, N, taps=4, dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.H, self.G, self.P, self.N = H, G, P, N
        self.sizes = (H * P, H * P + 2 * G * N, H)
        rand = lambda *n: torch.randn(*n, generator=gen, device=device) * n[0] ** -0.5  # noqa: E731
        self.w_in = rand(width, sum(self.sizes)).to(dtype)
        self.w_out = rand(H * P, width).to(dtype)
        self.w_conv = 0.5 * rand(taps, self.sizes[1]).t().contiguous()
        self.b_conv = torch.zeros(self.sizes[1], device=device)
        # decay rates 1 .. 16, step sizes 1e-3 .. 1e-1 before the token's own part
        self.A_log = torch.linspace(0.0, 2.77, H, device=device)
        self.dt_bias = torch.log(torch.expm1(torch.logspace(-3, -1, H, device=device)))
        self.skip = torch.ones(H, device=device)
        self.gamma = torch.ones(N, device=device)
        self.freqs = 1e4 ** (-torch.arange(N // 2, device=device) / (N // 2))

    def _project(self, u):
        return (u @ self.w_in).split(self.sizes, dim=-1)

    def _split(self, xbc, pos):
        x, Bm, Cm = xbc.split((self.H * self.P, self.G * self.N, self.G * self.N), dim=-1)
        Cm, Bm = lr.head_norm_rope(Cm, Bm, self.G, gamma_q=self.gamma, gamma_k=self.gamma, freqs=self.freqs, pos=pos)
        return x, Bm, Cm

    def _finish(self, y):
        return lr.group_norm_act(y, self.H) @ self.w_out

    def prompt(self, u, lens=None):
        """u (B, L, width), row b valid to lens[b]; returns (out, (inputs of the taps, state))."""
        B, L, _ = u.shape
        z, xbc, dt = self._project(u)
        xbc, taps = lr.causal_conv(xbc, self.w_conv, bias=self.b_conv, lens=lens)
        pos = torch.arange(L, dtype=torch.int32, device=u.device).expand(B, L).contiguous()
        x, Bm, Cm = self._split(xbc, pos)
        y, S = lr.selective_heads(x, dt, Bm, Cm, self.A_log, self.H, G=self.G, z=z, Dskip=self.skip,
                                  dt_bias=self.dt_bias, lens=lens)
        return self._finish(y), (taps, S)

    def token(self, u, pos, states):
        """u (B, width) at positions pos (B,); the states are updated in place; returns out."""
        taps, S = states
        z, xbc, dt = self._project(u)
        xbc, _ = lr.causal_conv_step(xbc, self.w_conv, bias=self.b_conv, state=taps, state_out=taps)
        x, Bm, Cm = self._split(xbc, pos)
        y, _ = lr.selective_heads_step(x, dt, Bm, Cm, self.A_log, self.H, G=self.G, z=z, Dskip=self.skip,
                                       dt_bias=self.dt_bias, S=S, S_out=S)
        return self._finish(y)


def run(batch=4, prompt=1024, tokens=32, width=1024, H=16, G=1, P=128, N=128, dtype=torch.bfloat16):
    """Times both phases and returns the largest differences of the tokens' outputs and of the
    state from one prompt call over everything, relative to the largest values."""
    layer = SelectiveLayer(width, H, G, P, N, dtype=dtype)
    gen = torch.Generator(device="cuda").manual_seed(1)
    u = torch.randn(batch, prompt + tokens, width, device="cuda", generator=gen).to(dtype)
    at = torch.arange(prompt, prompt + tokens + 1, dtype=torch.int32, device="cuda")
    whole, (_, S_whole) = layer.prompt(u)
    layer.token(u[:, 0], at[0].expand(batch).contiguous(), layer.prompt(u[:, :prompt])[1])   # warm-up
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    torch.cuda.synchronize()
    ev[0].record()
    _, states = layer.prompt(u[:, :prompt])
    ev[1].record()
    outs = [layer.token(u[:, prompt + i], at[i].expand(batch).contiguous(), states) for i in range(tokens)]
    ev[2].record()
    lr.check_status()
    torch.cuda.synchronize()
    print(f"prompt of {batch} x {prompt}: {ev[0].elapsed_time(ev[1]):.3f} ms, "
          f"a token of {batch} rows: {ev[1].elapsed_time(ev[2]) / max(tokens, 1):.3f} ms")
    far = lambda a, b: float((a.float() - b.float()).abs().max() / b.float().abs().max())  # noqa: E731
    e_state = far(states[1], S_whole)
    e_out = far(torch.stack(outs, 1), whole[:, prompt:]) if tokens else 0.0
    print(f"tokens against one call over all {prompt + tokens} steps: outputs {e_out:.1e}, state {e_state:.1e}")
    return e_out, e_state


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--batch", type=int, default=4)
    p.add_argument("--prompt", type=int, default=1024)
    p.add_argument("--tokens", type=int, default=32)
    a = p.parse_args()
    run(a.batch, a.prompt, a.tokens)
