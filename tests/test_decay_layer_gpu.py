"""The example layer: prompt, then tokens, against one call over the whole
sequence, and against the oracle's recurrence with the same projections."""
import importlib.util
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

EXAMPLE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "decay_attn_layer.py")


def _example():
    from selective_state_space_chunked_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("decay_attn_layer", EXAMPLE)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


# Both sides share every input, so they differ by roundings alone.  fp32: the sums
# of about 100 terms taken in another order, 100 * 2^-24 = 6e-6, with room 1e-4.
# bf16: the projections may round differently for other row counts (2^-8 each), and
# the norm divides a head's output by its own spread: a readout that happens to be a
# tenth of its usual size raises that head's error to 10 * 2^-8 = 4e-2, with room 6e-2;
# the fp32 state sees inputs with a relative difference of 2^-8 at most.
@pytest.mark.parametrize("dtype,tol_o,tol_s", [(torch.float32, 1e-4, 1e-4), (torch.bfloat16, 6e-2, 1e-2)])
@pytest.mark.parametrize("prompt", [1, 130])
def test_tokens_continue_the_prompt(dtype, tol_o, tol_s, prompt):
    e_out, e_state = _example().run(batch=3, prompt=prompt, tokens=5, width=256, H=8, Hk=2, dk=64, dv=32, dtype=dtype)
    assert e_out <= tol_o and e_state <= tol_s


def test_layer_against_the_oracle():
    import oracle
    m = _example()
    layer = m.DecayAttnLayer(128, 4, 2, 32, 64, torch.float32)
    x = torch.randn(2, 75, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    lens = torch.tensor([75, 31], device="cuda")
    out, S = layer.prompt(x, lens=lens)
    q, k, v, z, g = (t.contiguous() for t in layer._project(x))
    o, Sr = oracle.decay_attn(q.cpu(), k.cpu(), v.cpu(), 4, Hk=2, a_log=layer.a_log.cpu(), g=g.cpu(),
                              lens=lens.cpu().to(torch.int32), scale=32 ** -0.5)
    n = oracle.group_norm_act(np.asarray(o, np.float32).reshape(150, 256), 4, gamma=layer.gamma.cpu(),
                              z=z.cpu().reshape(150, 256))
    ref = np.asarray(n, np.float64).reshape(2, 75, 256) @ layer.w_out.double().cpu().numpy()
    # rows past a length have o = 0 and so a norm of 0
    assert float(out[1, 31:].abs().max()) == 0.0
    # fp32 throughout, sums of up to 256 terms: 256 * 2^-24 = 1.5e-5, with room 1e-4
    assert np.max(np.abs(out.double().cpu().numpy() - ref)) <= 1e-4 * np.max(np.abs(ref))
    assert np.max(np.abs(S.double().cpu().numpy() - np.asarray(Sr, np.float64))) <= 1e-4 * np.max(np.abs(Sr))
