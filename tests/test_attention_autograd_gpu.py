"""GPU tests of linear attention's autograd wrapper with gradients as a training graph delivers them: dense, but anywhere in
memory."""
import numpy as np
import pytest

from synth import round_to_bf16
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mss():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_06_amd as m
    m.load_library()
    return m


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ahead", [1, 3])
def test_gradients_behind_an_odd_number_of_elements(mss, ahead, dtype):
    """out and last_state that went through a concatenation have views of its gradient, at any element."""
    import torch
    rng = np.random.default_rng(ahead)
    draw = lambda *s: dev(round_to_bf16(rng.standard_normal(s).astype(np.float32)), dtype)  # noqa: E731
    q, k, v, dout = draw(2, 37, 3, 32), draw(2, 37, 3, 32), draw(2, 37, 3, 48), draw(2, 37, 3, 48)
    S, E = (dev(rng.standard_normal((2, 3, 32, 48)).astype(np.float32)) for _ in range(2))
    rate = dev(np.array([0.01, 0.1, 1.0], dtype=np.float32))
    leaves = [t.clone().requires_grad_() for t in (q, k, v, S)]
    out, last = mss.LinearAttentionFunction.apply(*leaves[:3], rate, 0.5, leaves[3])
    a = torch.cat([torch.zeros(ahead, device="cuda", dtype=out.dtype), out.flatten()])
    b = torch.cat([torch.zeros(ahead, device="cuda"), last.flatten()])
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    da[ahead:], db[ahead:] = dout.flatten(), E.flatten()
    torch.autograd.backward([a, b], [da, db])
    g = mss.linear_attention_bwd(q, k, v, rate, dout, scale=0.5, initial_state=S, dlast_state=E, return_dinitial_state=True)
    for t, n in zip(leaves, ("dq", "dk", "dv", "dinitial_state")):
        assert torch.equal(t.grad, g[n]), n
