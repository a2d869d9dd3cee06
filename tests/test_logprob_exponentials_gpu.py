"""GPU tests of the log probabilities' exponentials far from a row's greatest logit.

Tolerances relative to the result, u = 2^-24, for a row whose greatest logit is 0 (d = x - m is x as it stands): e^d is one
exp2 (2 u) and one corrected product (1 u), whatever d; the sum of the row in a lane's 8 + 2 n terms, n = vocab / 4096 + 1,
and 64 bits from there; 1 / s rounds once, the product once, g and its sign none: (3 + 8 + 2 n + 2 + 2) u.  Without the
correction d log2 e alone, rounded, is up to 44 u off at d = -80."""
import numpy as np
import pytest

import oracle
from tests.gpu_helpers import dev, host64

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


def rows(V, low, seed):
    rng = np.random.default_rng(seed)
    x = rng.uniform(low, 0.0, (4, V)).astype(np.float32)
    x[:, 1] = 0.0
    return x


@pytest.mark.parametrize("V", [64, 1000, 20001, 50280])
@pytest.mark.parametrize("low", [-5.0, -40.0, -84.0])
def test_gradients_of_improbable_tokens(mss, V, low):
    import torch
    x, n = rows(V, low, V), V / 4096 + 1
    t = torch.ones(4, dtype=torch.int32, device="cuda")
    saved = mss.token_logprobs_save(dev(x), t)[2]
    d = host64(mss.token_logprobs_bwd(dev(x), t, saved, torch.ones(4, device="cuda")))
    ref, _ = oracle.token_logprobs_bwd(x, np.ones(4, np.int32), np.ones(4))
    off = np.maximum(np.abs(d - ref) - 2.0 ** -126, 0.0) / np.abs(ref)  # (under 2^-126 fp32 has no more than that)
    off[:, 1] = 0.0  # the token's own: 1 - p, a difference
    assert off.max() <= (15 + 2 * n) * U, float(off.max() / U)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sum_of_many_equal_logits(mss, dtype):
    """One logit of 0 and 65535 that are equal: every term of the sum has the same error, which no average takes away.
    log s is (1 - 1 / s) of that and the lanes' (8 + 2 n) u off, the result rounds once."""
    import torch
    V = 65536
    for low in (-10.25, -11.0, -11.5, -12.75, -13.5, -9.625):
        x = np.full((1, V), low, dtype=np.float32)
        x[0, 777] = 0.0
        lp, en = mss.token_logprobs(dev(x, dtype), torch.tensor([777], dtype=torch.int32, device="cuda"))
        o = oracle.token_logprobs(x, np.array([777]))
        n = V / 4096 + 1
        assert abs(float(lp[0]) - o["logprobs"][0]) <= (3 + 8 + 2 * n) * U + U * abs(o["logprobs"][0])
        assert abs(float(en[0]) - o["entropy"][0]) <= 2 * (3 + 8 + 2 * n) * U * (1 + abs(low)) + U * o["entropy"][0]


def test_masked_rows_infinities_and_nan(mss):
    """The correction of what is not finite: -inf has no part in a row, +inf and NaN make it NaN."""
    import torch
    x = np.random.default_rng(3).standard_normal((5, 700)).astype(np.float32)
    x[0, 5:] = -np.inf
    x[1] = -np.inf
    x[2, 9] = np.nan
    x[3, 9] = np.inf
    x[4, 7:] = -3.4e38
    t = torch.zeros(5, dtype=torch.int32, device="cuda")
    lp, en, saved = mss.token_logprobs_save(dev(x), t)
    o = oracle.token_logprobs(x, np.zeros(5, np.int32))
    for got, ref in ((lp, o["logprobs"]), (en, o["entropy"])):
        g = host64(got)
        assert np.array_equal(np.isnan(g), np.isnan(ref)) and np.array_equal(np.isinf(g), np.isinf(ref))
        f = np.isfinite(ref)
        assert np.all(np.abs(g - ref)[f] <= 32 * U * (1 + np.abs(ref[f])))
    d = host64(mss.token_logprobs_bwd(dev(x), t, saved, torch.ones(5, device="cuda"), torch.ones(5, device="cuda")))
    assert not d[0, 5:].any() and not d[1].any() and np.isnan(d[2]).all() and np.isnan(d[3, 9])
    ref, M = oracle.token_logprobs_bwd(x, np.zeros(5, np.int32), np.ones(5), np.ones(5))
    for r in (0, 4):
        assert np.all(np.abs(d[r] - ref[r]) <= 40 * U * (M[r] + 1e-3))
