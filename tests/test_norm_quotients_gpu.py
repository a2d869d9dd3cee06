"""GPU tests of the 8-bit norm's quotients: out is the fp32 quotient (z rstd weight) / scale rounded to nearest even, also
where that lies on or next to the middle between two 8-bit values.

Rows of +-1 without eps have rstd 1 exactly, so that z rstd weight is the weight as it stands; scale is the fp32 quotient
of a group's greatest weight and 448.  Every step of the definition is then one fp32 operation, which numpy does too: the
bits have to agree, without a tolerance."""
import numpy as np
import pytest

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


def weights(rng, W, group):
    """Weights whose quotients are the middles between neighbouring 8-bit values, or the fp32 values next to those."""
    middles = np.array([(8 + k + 0.5) * 2.0 ** e for e in range(-9, 6) for k in range(8) if (8 + k + 0.5) * 2.0 ** e < 448])
    w = np.empty(W, dtype=np.float32)
    for i in range(0, W, group):
        n = min(group, W - i)
        most = np.float32(rng.uniform(1.0, 2.0))
        scale = most / np.float32(448)
        v = np.float32(scale * rng.choice(middles, n))
        step = rng.integers(-1, 2, n)
        w[i:i + n] = np.where(step < 0, np.nextafter(v, np.float32(0)), np.where(step > 0, np.nextafter(v, np.float32(9)), v))
        w[i] = most
    return w


@pytest.mark.parametrize("group", [None, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("W", [256, 4096, 16384])
def test_quotients_next_to_the_middle(mss, W, dtype, group):
    import torch
    rng = np.random.default_rng(W)
    for _ in range(4):
        w = weights(rng, W, group or W)
        x = rng.choice(np.array([-1.0, 1.0], dtype=np.float32), (3, W))
        assert bool((mss.rms_norm_fwd_save(dev(x, dtype), dev(w), eps=0.0)[2] == 1.0).all())
        q, scales, _ = mss.rms_norm_fwd_e4m3(dev(x, dtype), dev(w), eps=0.0, group=group)
        n = group or W
        want = np.repeat(np.stack([w[i:i + n].max() / np.float32(448) for i in range(0, W, n)]), n)[:W]
        assert np.array_equal(np.repeat(scales.cpu().numpy(), n, 1)[:, :W], np.tile(want, (3, 1)))
        quotient = x * (w / want)
        assert quotient.dtype == np.float32
        assert torch.equal(q.cpu().view(torch.uint8), torch.from_numpy(quotient).to(torch.float8_e4m3fn).view(torch.uint8))
