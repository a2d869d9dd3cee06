"""GPU tests of the RMS norm's dweight: a sum over many rows whose small terms count beside large ones.

Rows of +-1 without eps have rstd 1 exactly: dweight is the sum of +-dout, products without a rounding.  The sum is held in
64 bits; a block's part of it is rounded to fp32, and the whole once more: u (sum of the parts' magnitudes) and u of the
result, 2 u = 2^-23 of it where all terms have one sign."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def mss():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_06_amd as m
    m.load_library()
    return m


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("R,W", [(163840, 256), (40000, 1024), (20000, 8192), (9000, 16384)])
def test_small_terms_behind_large_ones(mss, R, W, residual):
    import torch
    g = torch.Generator(device="cuda").manual_seed(R)
    x = torch.randint(0, 2, (R, W), generator=g, device="cuda").float() * 2 - 1
    d = torch.full((R, W), 1.5 * 2.0 ** -25, device="cuda")
    d[:2560] = 1.0
    rstd = torch.ones(R, device="cuda")
    w = torch.ones(W, device="cuda")
    got = mss.rms_norm_bwd(x, w, rstd, x * d, dresidual_out=x if residual else None)["dweight"].double()
    want = d.double().sum(0)
    assert bool(((got - want).abs() <= 2 * U * want).all()), float(((got - want).abs() / want).max() / U)


def test_random_terms(mss):
    """Terms of both signs, against the sum in 64 bits: u of the parts and of the result."""
    import torch
    R, W = 6123, 2049
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(0, 2, (R, W), generator=g, device="cuda").float() * 2 - 1
    d = torch.randn(R, W, generator=g, device="cuda")
    got = mss.rms_norm_bwd(x, torch.ones(W, device="cuda"), torch.ones(R, device="cuda"), d)["dweight"].double()
    t = (x.double() * d.double())
    assert bool(((got - t.sum(0)).abs() <= 2 * U * t.abs().sum(0)).all())
