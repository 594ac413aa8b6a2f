"""The example layer of the selective scan with heads: a prompt, then tokens, against one
call over the whole sequence (test_layer_helpers_gpu has the operators together against the
oracle)."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

EXAMPLE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "selective_layer.py")


# Both sides share every input, so they differ by roundings alone.  fp32: sums of up to 256
# terms taken in another order, 256 * 2^-24 = 1.5e-5, through norms: 1e-4.  bf16: projections,
# convolution and norm round by 2^-8 each, possibly otherwise for other row counts; B and C
# carry that into the state (three roundings of independent terms, 3 * 2^-8 = 1.2e-2), and the
# norm divides a head's output by its own spread, which raises a small head's error several
# times: 6e-2.
@pytest.mark.parametrize("dtype,tol_o,tol_s", [(torch.float32, 1e-4, 1e-4), (torch.bfloat16, 6e-2, 1.2e-2)])
@pytest.mark.parametrize("prompt", [1, 130])
def test_tokens_continue_the_prompt(dtype, tol_o, tol_s, prompt):
    from selective_state_space_chunked_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("selective_layer", EXAMPLE)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    e_out, e_state = mod.run(batch=3, prompt=prompt, tokens=5, width=256, H=8, G=2, P=64, N=32, dtype=dtype)
    assert e_out <= tol_o and e_state <= tol_s
