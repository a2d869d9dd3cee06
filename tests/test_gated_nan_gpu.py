"""GPU tests of the gated scan on values that are no numbers: a NaN (in an input, a gate, the outer
gradient, a state) reaches exactly the outputs and gradients whose formula it stands in, and an
infinite gate is its sigmoid's limit."""
import numpy as np
import pytest

import oracle
from tests.gpu_helpers import host64
from tests.test_gated_gpu import inputs, limits, mss, upload  # noqa: F401

pytestmark = pytest.mark.gpu


def run(m, c):
    t = upload(c)
    out, last, saved = m.gated_scan_fwd_save(t["x"], t["f"], t["i"], t["rate"], initial_state=t["h0"],
                                             seq_lens=t["lens"])
    g = m.gated_scan_bwd(t["x"], t["f"], t["i"], t["rate"], t["dout"], seq_lens=t["lens"], saved_states=saved,
                         dlast_state=t["dlast"], return_dinitial_state=True)
    return {"out": out, "last": last, "dx": g["dx"], "dfgate": g["dfgate"], "digate": g["digate"],
            "dh0": g["dinitial_state"], "drate": g["drate"]}


# rates below 1/4 and above take different code; rows of whole vectors, others, and several waves to a row
@pytest.mark.parametrize("L,dtype", [(40, "f32"), (1303, "f32"), (1304, "bf16"), (5000, "bf16"), (70001, "f32")])
@pytest.mark.parametrize("lo,hi", [(0.9, 0.999), (0.2, 0.7)])
@pytest.mark.parametrize("name", ["x", "f", "i", "dout", "h0", "dlast"])
def test_a_nan_reaches_what_it_stands_in(mss, name, L, dtype, lo, hi):  # noqa: F811
    c = inputs(1, 3, L, dtype, L, False, True, lo, hi)
    at = (L * 3 // 5, 0, L - 1)
    for d, k in enumerate(at):  # a channel each
        c[name][(0, d, k) if c[name].ndim == 3 else (0, d)] = np.nan
    got = run(mss, c)
    with np.errstate(invalid="ignore"):
        out, last, _ = oracle.gated_scan(c["x"], c["f"], c["i"], c["rate"], c["h0"])
        g = oracle.gated_scan_bwd(c["x"], c["f"], c["i"], c["rate"], c["dout"], c["h0"], None, c["dlast"])
    want = dict(g, out=out, last=last)
    for n, v in got.items():
        np.testing.assert_array_equal(np.isnan(host64(v)), np.isnan(want[n]), err_msg=f"{name} -> {n}")


@pytest.mark.parametrize("rate", [0.1, 0.3])
def test_a_closed_gate_passes_nothing(mss, rate):  # noqa: F811
    """fgate at -inf: a = 1 and the input's weight sqrt(1 - a^2) is 0, so the state is held and x and igate get
    exactly no gradient at that step; at +inf it is an open gate."""
    c = inputs(1, 2, 700, "f32", 3, False, True)
    c["rate"][:] = rate
    c["f"][0, 0, ::3] = -np.inf
    c["f"][0, 1, ::3] = np.inf
    got = {n: host64(v) for n, v in run(mss, c).items()}
    assert all(np.isfinite(v).all() for v in got.values())
    assert not got["dx"][0, 0, ::3].any() and not got["digate"][0, 0, ::3].any() and not got["dfgate"][0, :, ::3].any()
    # held: exactly, but where a step is the first of a lane's eight, which starts from a fold of the steps before in
    # another order than the walk that gave the step before it: there both are the same exact state to within the
    # forward's limit
    t = np.arange(3, 700, 3)
    now, then = got["out"][0, 0, t], got["out"][0, 0, t - 1]
    walked = t % 8 != 0
    np.testing.assert_array_equal(now[walked], then[walked])
    M, _, _ = oracle.gated_scan(np.abs(c["x"]), c["f"], c["i"], c["rate"], np.abs(c["h0"]))
    assert np.all(np.abs(now - then) <= 2 * limits(c, M, M)[0, 0, t])
    # the open channel: as with a gate so far open that its sigmoid is 1 in fp32
    c["f"][0, 1, ::3] = 200.0
    same = {n: host64(v) for n, v in run(mss, c).items()}
    for n in got:
        np.testing.assert_array_equal(got[n], same[n], err_msg=n)
