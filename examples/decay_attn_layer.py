"""A decayed linear-attention layer for serving: a prompt in one call, then one
token per call from the state that the prompt left.

    python examples/decay_attn_layer.py [--batch 4] [--prompt 1024] [--tokens 32]

The layer projects its input to queries, keys, values, an output gate and a log
decay per head, runs the attention, normalises each head's output, multiplies it
by the gate and projects back:

    o   = decay_attn(q, k, v, g)           (prompt)
        = decay_attn_step(q, k, v, g, S)   (token)
    out = (group_norm(o) silu(z)) W_out

The projections are plain matrix products.  The script prints the times of both
phases and how far the tokens' outputs are from those of one prompt call over the
whole sequence.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from selective_state_space_chunked_gb300 import binding as lr  # noqa: E402


class DecayAttnLayer:
    """H value heads of dv channels over Hk shared key heads of dk channels; the
    decay of head h at a token is exp(a_log[h] + g), both at most 0."""

    def __init__(self, width, H, Hk, dk, dv, dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.sizes = (Hk * dk, Hk * dk, H * dv, H * dv, H)
        self.H, self.Hk, self.dk, self.dv = H, Hk, dk, dv
        rand = lambda *n: torch.randn(*n, generator=gen, device=device) * n[0] ** -0.5  # noqa: E731
        self.w_in = rand(width, sum(self.sizes)).to(dtype)
        self.w_out = rand(H * dv, width).to(dtype)
        # half-lives from a few tokens to a thousand, spread over the heads
        self.a_log = -torch.logspace(-3, 0, H, device=device) * 0.69
        self.gamma = torch.ones(H * dv, device=device)

    def _project(self, x):
        q, k, v, z, g = (x @ self.w_in).split(self.sizes, dim=-1)
        return q, k, v, z, torch.nn.functional.logsigmoid(g.float() + 4.0).to(x.dtype)

    def _finish(self, o, z):
        return lr.group_norm_act(o, self.H, gamma=self.gamma, z=z) @ self.w_out

    def prompt(self, x, lens=None, S=None):
        """x (B, L, width), row b valid to lens[b]; returns (out, state)."""
        q, k, v, z, g = self._project(x)
        o, S = lr.decay_attn(q, k, v, self.H, Hk=self.Hk, a_log=self.a_log, g=g, S0=S, lens=lens,
                             scale=self.dk ** -0.5)
        return self._finish(o, z), S

    def token(self, x, S):
        """x (B, width); the state S is updated in place; returns out."""
        q, k, v, z, g = self._project(x)
        o, _ = lr.decay_attn_step(q, k, v, self.H, Hk=self.Hk, a_log=self.a_log, g=g, S=S, S_out=S,
                                  scale=self.dk ** -0.5)
        return self._finish(o, z)


def run(batch=4, prompt=1024, tokens=32, width=1024, H=16, Hk=4, dk=128, dv=128, dtype=torch.bfloat16):
    """Times both phases and returns the largest difference between the tokens'
    outputs and one prompt call over everything, relative to the largest output."""
    layer = DecayAttnLayer(width, H, Hk, dk, dv, dtype)
    x = torch.randn(batch, prompt + tokens, width, device="cuda").to(dtype)
    whole, S_whole = layer.prompt(x)
    layer.token(x[:, 0], layer.prompt(x[:, :prompt])[1])   # warm-up
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    torch.cuda.synchronize()
    ev[0].record()
    _, S = layer.prompt(x[:, :prompt])
    ev[1].record()
    outs = [layer.token(x[:, prompt + i], S) for i in range(tokens)]
    ev[2].record()
    lr.check_status()
    torch.cuda.synchronize()
    print(f"prompt of {batch} x {prompt}: {ev[0].elapsed_time(ev[1]):.3f} ms, "
          f"a token of {batch} rows: {ev[1].elapsed_time(ev[2]) / max(tokens, 1):.3f} ms")
    far = lambda a, b: float((a.float() - b.float()).abs().max() / b.float().abs().max())  # noqa: E731
    e_state = far(S, S_whole)
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
