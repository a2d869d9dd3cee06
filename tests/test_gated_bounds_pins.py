"""The limits of the gated scan's GPU tests, without a GPU: their values are the oracle's, and they tell a
right result from a wrong one."""
import numpy as np
import pytest

import oracle
from tests.test_gated_bounds_gpu import CASES, carried, make, worth


@pytest.mark.parametrize("lens", [False, True])
def test_values_are_the_oracles(lens):
    c = make(2, 3, 700, "f32", 1, False, lens)
    lim, parts = carried(c, 100)
    out, last, before = oracle.gated_scan(c["x"], c["f"], c["i"], c["rate"], c["h0"], c["lens"])
    g = oracle.gated_scan_bwd(c["x"], c["f"], c["i"], c["rate"], c["dout"], c["h0"], c["lens"], c["dlast"])
    want = dict(out=out, last=last, saved=before[..., ::512], **{n: g[n] for n in ("dx", "dfgate", "digate", "dh0", "drate")})
    assert want.keys() == lim.keys()
    for n, r in want.items():
        assert np.abs(lim[n][0] - r).max() < 1e-10 * (1 + np.abs(r).max()), n
    assert np.abs(parts.sum((0, 2)) - g["drate"]).max() < 1e-10 * np.abs(parts).sum()


@pytest.mark.parametrize("case", CASES)
def test_limits_are_worth_something(case):
    B, D, L, dtype, lens, cuts = case
    for sign in (True, False):
        c = dict(make(B, D, L, dtype, B + D + L, sign, lens), sign=sign, cuts=cuts)
        worth(c, *carried(c, cuts))
