"""GPU tests of a selected score's own accuracy: the normaliser, whose sum of exponentials is fp32, and
scores at the end of fp32's range.

u = 2^-24.  A term e^(v - m) is off by (3 |v - m| + 2) u: the difference, the constant log2 e, their product, exp2.
Under the softmax's own weights the mean of |v - m| is at most ln V (the entropy is at most ln V), once for a
tile's reference and once for the rescaling to the row's: 6 ln V.  A lane adds a tile of eight and, of the tiles
of its wave (V / 4096, at most, and one), one sum and one rescaling (3 u) each: V / 1024 + 16.  With 16 more for
the joins: the sum is off by (6 ln V + V / 1024 + 32) u of itself, its logarithm by the same."""
import numpy as np
import pytest

import oracle
from synth import round_to_bf16
from tests.gpu_helpers import dev, record_margin
from tests.test_gated_gpu import mss  # noqa: F401

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def near_zero(x):
    """Scores (fp32) for which every beam's best continuation comes out near 0, where fp32 shows the normaliser's
    own error."""
    x = x.astype(np.float64)
    top = x.max(-1)
    return np.log(np.exp(x - top[..., None]).sum(-1)).astype(np.float32)


@pytest.mark.parametrize("V,dtype", [(5, "f32"), (1000, "bf16"), (32768, "bf16"), (50001, "f32"), (128007, "f32"),
                                     (128008, "bf16")])
@pytest.mark.parametrize("how", ["normal", "rising", "flat"])
def test_the_normalisers_error(mss, V, dtype, how):  # noqa: F811
    rng = np.random.default_rng(V)
    x = (2.5 * rng.standard_normal((3, 8, V))).astype(np.float32)
    if how == "rising":
        x = np.sort(x, -1)
    if how == "flat":
        x = (1e-3 * x).astype(np.float32)
    x = round_to_bf16(x) if dtype == "bf16" else x
    s = near_zero(x)
    got = mss.beam_select(dev(x, dtype), dev(s), k=8)
    want = oracle.beam_select(x, s, k=8)
    bound = (6 * np.log(V) + V / 1024 + 32) * U
    err = np.abs(got[0].cpu().numpy().astype(np.float64) - want[0])
    err = err[np.isfinite(want[0])]
    record_margin(f"beam normaliser {V} {dtype} {how}", err.max() / (bound + np.abs(want[0][np.isfinite(want[0])]).max() * U))
    assert np.all(err <= bound + np.abs(want[0][np.isfinite(want[0])]) * U)


def test_beams_that_differ_by_less_than_the_normalisers_error(mss):  # noqa: F811
    """The same logits in another order tie by the definition; each beam's own candidates come in their order, and the
    beams' interleave by rounding, so that at every rank the score is the definition's."""
    rng = np.random.default_rng(1)
    row = (2.5 * rng.standard_normal(20000)).astype(np.float32)
    x = np.stack([row, row[::-1], rng.permutation(row), row])[None]
    s = np.zeros((1, 4), np.float32)
    got = mss.beam_select(dev(x), dev(s), k=32)
    want = oracle.beam_select(x, s, k=32)
    bound = (6 * np.log(20000) + 20000 / 1024 + 32) * U
    assert np.all(np.abs(got[0].cpu().numpy() - want[0]) <= bound + np.abs(want[0]) * U)
    p, t = got[1].cpu().numpy()[0], got[2].cpu().numpy()[0]
    for beam in range(4):
        own = np.argsort(-x[0, beam], kind="stable")
        mine = t[p == beam]
        assert 7 <= len(mine) <= 9
        np.testing.assert_array_equal(mine, own[:len(mine)])
    # beam 3 is a copy of beam 0, with the same normaliser to the bit: 0 comes first
    first, copy = np.flatnonzero(p == 0), np.flatnonzero(p == 3)
    assert np.all(first[:7] < copy[:7])


def test_scores_below_fp32s_range(mss):  # noqa: F811
    """Lowest-value scores and lowest-value logits add up past fp32's range: written as -inf, and no continuation
    of the step after."""
    low = np.finfo(np.float32).min
    x = np.array([[[1.0, 2.0, low], [low, 3.0, low]]], np.float32)
    s = np.array([[-1.0, low]], np.float32)
    got = mss.beam_select(dev(x), dev(s), k=6)
    score, parent, token = (v.cpu().numpy()[0] for v in got)
    assert token[:2].tolist() == [1, 0] and parent[:2].tolist() == [0, 0]
    assert (parent[2], token[2]) in ((0, 2), (1, 1)) and score[2] == low and score[3] == low  # equal in fp32
    assert np.all(score[4:] == -np.inf) and parent[4:].tolist() == [1, 1] and token[4:].tolist() == [0, 2]
    again = mss.beam_select(dev(np.zeros((1, 6, 3), np.float32)), got[0], k=18)
    assert not np.isin(again[1].cpu().numpy()[0][np.isfinite(again[0].cpu().numpy()[0])], (4, 5)).any()
