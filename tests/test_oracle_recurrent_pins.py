"""Pins of the fp64 definitions of the gated scan, the conv's gradients and beam selection: closed
forms, hand computed cases, and every gradient against central differences of the forward.

Differences: with step e = 1e-5 on values of order 1 the central difference is off by the third
derivative times e^2 / 6 (about 1e-10 here) plus the rounding of the loss, about 2^-53 * 100 / e =
1e-9; the tolerance 2e-6 is far above both and far below any wrong term."""
import numpy as np
import pytest

import oracle


def _scan_inputs(seed, B=2, D=3, L=7):
    rng = np.random.default_rng(seed)
    x, f, i, dout = (rng.standard_normal((B, D, L)) for _ in range(4))
    return x, f, i, rng.uniform(0.05, 1.5, D), rng.standard_normal((B, D)), dout, rng.standard_normal((B, D))


def test_gated_scan_one_step_and_open_gates():
    x, f, i, rate, h0, _, _ = _scan_inputs(0, L=1)
    out, last, _ = oracle.gated_scan(x, f, i, rate, h0)
    r = 1 / (1 + np.exp(-f[..., 0]))
    a = np.exp(-rate * r)
    want = a * h0 + np.sqrt(1 - a * a) / (1 + np.exp(-i[..., 0])) * x[..., 0]
    np.testing.assert_allclose(out[..., 0], want, rtol=1e-12)
    np.testing.assert_array_equal(last, out[..., 0])
    # gates fully open, constant input: h_t = b (1 - a^t) / (1 - a), b = sqrt(1 - a^2)
    B, D, L = 1, 2, 20
    big = np.full((B, D, L), 60.0)
    rate = np.array([0.3, 1.1])
    out, _, _ = oracle.gated_scan(np.ones((B, D, L)), big, big, rate)
    a = np.exp(-rate)[:, None]
    t = np.arange(1, L + 1)
    np.testing.assert_allclose(out[0], np.sqrt(1 - a * a) * (1 - a ** t) / (1 - a), rtol=1e-12)


def test_gated_scan_lengths_and_chunks():
    x, f, i, rate, h0, _, _ = _scan_inputs(1, B=3, L=9)
    lens = [0, 4, 9]
    out, last, _ = oracle.gated_scan(x, f, i, rate, h0, seq_lens=lens)
    for b, n in enumerate(lens):
        o, l, _ = oracle.gated_scan(x[b:b + 1, :, :n], f[b:b + 1, :, :n], i[b:b + 1, :, :n], rate, h0[b:b + 1])
        np.testing.assert_array_equal(out[b, :, :n], o[0])
        assert not out[b, :, n:].any()
        np.testing.assert_array_equal(last[b], l[0])
    o1, l1, _ = oracle.gated_scan(x[..., :4], f[..., :4], i[..., :4], rate, h0)
    o2, l2, _ = oracle.gated_scan(x[..., 4:], f[..., 4:], i[..., 4:], rate, l1)
    whole, lw, _ = oracle.gated_scan(x, f, i, rate, h0)
    np.testing.assert_array_equal(np.concatenate([o1, o2], -1), whole)
    np.testing.assert_array_equal(l2, lw)
    np.testing.assert_allclose(oracle.gated_state_update(h0, x[..., 0], f[..., 0], i[..., 0], rate), whole[..., 0],
                               rtol=1e-14)


def _differences(loss, arrays, grads, tol=2e-6, e=1e-5):
    for name, arr in arrays.items():
        flat, g = arr.reshape(-1), grads[name].reshape(-1)
        for j in range(flat.size):
            keep = flat[j]
            flat[j] = keep + e
            up = loss()
            flat[j] = keep - e
            down = loss()
            flat[j] = keep
            assert abs((up - down) / (2 * e) - g[j]) < tol * max(1.0, abs(g[j])), (name, j, (up - down) / (2 * e), g[j])


@pytest.mark.parametrize("lens", [None, [0, 5], [7, 1]])
def test_gated_scan_gradients_against_differences(lens):
    x, f, i, rate, h0, dout, dlast = _scan_inputs(2)

    def loss():
        out, last, _ = oracle.gated_scan(x, f, i, rate, h0, seq_lens=lens)
        return float((out * dout).sum() + (last * dlast).sum())

    g = oracle.gated_scan_bwd(x, f, i, rate, dout, h0, seq_lens=lens, dlast=dlast)
    _differences(loss, dict(dx=x, dfgate=f, digate=i, drate=rate, dh0=h0), g)
    for n in ("dx", "dfgate", "digate", "drate", "dh0"):
        assert np.all(np.abs(g[n]) <= g["m_" + n] * (1 + 1e-12) + 1e-300), n


def test_gated_scan_closed_forget_gate_is_finite():
    """Where the forget gate is so far closed that rate r is 0 in fp64, a = 1 and nothing enters:
    the state is held and every gradient is finite (the limit of rate r -> 0)."""
    x, f, i, rate, h0, dout, _ = _scan_inputs(3)
    f[..., 2] = -800.0
    out, _, _ = oracle.gated_scan(x, f, i, rate, h0)
    np.testing.assert_array_equal(out[..., 2], out[..., 1])
    g = oracle.gated_scan_bwd(x, f, i, rate, dout, h0)
    assert all(np.isfinite(v).all() for v in g.values())


@pytest.mark.parametrize("K,L,silu,with_state", [(4, 6, True, True), (4, 2, True, True), (3, 5, False, True),
                                                 (2, 1, True, False), (1, 4, True, False), (4, 0, True, True)])
def test_conv_gradients_against_differences(K, L, silu, with_state):
    rng = np.random.default_rng(K * 10 + L)
    B, D = 2, 3
    x, dout = rng.standard_normal((B, D, L)), rng.standard_normal((B, D, L))
    w, b = rng.standard_normal((D, K)), rng.standard_normal(D)
    st = rng.standard_normal((B, D, K - 1)) if with_state else None
    dfin = rng.standard_normal((B, D, K - 1)) if with_state else None

    def loss():
        out, fin = oracle.causal_conv1d(x, w, b, state=st, silu=silu)
        return float((out * dout).sum() + (0.0 if dfin is None else (fin * dfin).sum()))

    g = oracle.causal_conv1d_bwd(x, w, dout, b, st, silu, dfin)
    arrays = dict(dx=x, dweight=w, dbias=b)
    if with_state:
        arrays["dstate"] = st
    _differences(loss, arrays, g)


def test_beam_select_by_hand():
    # beam 0: p = (1/2, 1/4, 1/4), beam 1: p = (1/8, 3/4, 1/8)
    logits = np.log(np.array([[[2.0, 1.0, 1.0], [1.0, 6.0, 1.0]]]))
    s, p, v, d = oracle.beam_select(logits, np.zeros((1, 2)), k=4)
    np.testing.assert_allclose(np.exp(s[0]), [0.75, 0.5, 0.25, 0.25], rtol=1e-12)
    assert p[0].tolist() == [1, 0, 0, 0] and v[0].tolist() == [1, 0, 1, 2] and not d.any()
    # one beam at its end: its single continuation keeps its score
    s, p, v, d = oracle.beam_select(logits, np.array([[0.0, -1.0]]), k=6, finished=np.array([[0, 1]]), end_token=2)
    assert p[0, :4].tolist() == [0, 1, 0, 0] and v[0, :4].tolist() == [0, 2, 1, 2] and d[0, :4].tolist() == [0, 1, 0, 1]
    assert np.all(s[0, 4:] == -np.inf) and not d[0, 4:].any()
    # nothing left: a row of -inf, a NaN logit, a beam that was never used
    gone = np.array([[[-np.inf] * 3, [np.nan, 1.0, 1.0]]])
    s, p, v, _ = oracle.beam_select(gone, np.array([[0.0, 0.0]]), k=3)
    assert v[0].tolist() == [1, 2, 0] and p[0].tolist() == [1, 1, 0] and s[0, 2] == -np.inf
    s, _, _, _ = oracle.beam_select(logits, np.array([[-np.inf, -np.inf]]))
    assert np.all(s == -np.inf)


def test_beam_reorder_takes_parents_and_keeps_bad_ones():
    st = np.arange(12.0).reshape(6, 2)
    got = oracle.beam_reorder(st, np.array([[2, 0, 0], [1, 7, -1]]))
    np.testing.assert_array_equal(got, st[[2, 0, 0, 4, 4, 5]])
