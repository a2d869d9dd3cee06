"""What the fp64 definitions of the RMS norm, linear attention and token log probabilities are pinned by: closed forms,
sums written out, and central differences of their own forwards.

A difference (f(x + e) - f(x - e)) / 2e with e = 1e-5 is off by e^2 f''' / 6, about 1e-10 for these values of size 1, and
by the rounding 1e-16 |f| / e, about 1e-10 for |f| up to 10: 1e-7 holds both with room."""
import numpy as np
import pytest

import oracle

E = 1e-5


def differences(f, x, at):
    got = []
    for i in at:
        hi, lo = x.copy(), x.copy()
        hi[i] += E
        lo[i] -= E
        got.append((f(hi) - f(lo)) / (2 * E))
    return np.array(got)


def some(x, rng, n=6):
    return [tuple(rng.integers(0, s) for s in x.shape) for _ in range(n)]


def agree(f, x, grad, rng):
    at = some(x, rng)
    want = differences(f, x, at)
    assert np.allclose([grad[i] for i in at], want, rtol=1e-6, atol=1e-7)


def test_norm_of_a_row_of_equal_values():
    out, rstd = oracle.rms_norm(np.full((1, 5), -3.0), np.arange(5.0), 7.0)
    assert np.allclose(rstd, 0.25) and np.allclose(out, -0.75 * np.arange(5.0))


def test_norm_gradients_are_differences():
    rng = np.random.default_rng(0)
    z, w, d, s = rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal((3, 7)), rng.standard_normal((3, 7))
    g = oracle.rms_norm_bwd(z, w, 1e-3, d, s)
    agree(lambda a: np.sum(d * oracle.rms_norm(a, w, 1e-3)[0]) + np.sum(s * a), z, g["dz"], rng)
    agree(lambda a: np.sum(d * oracle.rms_norm(z, a, 1e-3)[0]), w, g["dweight"], rng)
    assert np.all(g["m_dz"] >= np.abs(g["dz"])) and np.all(g["m_dweight"] >= np.abs(g["dweight"]))


def attention_inputs(rng, B=2, L=5, H=6, heads=(2, 3, 6), K=3, V=4):
    n = rng.standard_normal
    return dict(q=n((B, L, heads[0], K)), k=n((B, L, heads[1], K)), v=n((B, L, heads[2], V)),
                rate=rng.uniform(0.01, 0.7, H), S0=n((B, H, K, V)), seq_lens=np.array([L, 3])[:B])


def test_attention_is_the_decayed_sum_over_pairs():
    rng = np.random.default_rng(1)
    c = attention_inputs(rng)
    out, last = oracle.linear_attention(c["q"], c["k"], c["v"], c["rate"], 0.7, c["S0"], c["seq_lens"])
    want = np.zeros_like(out)
    for b in range(2):
        for h in range(6):
            a = np.exp(-c["rate"][h])
            for t in range(c["seq_lens"][b]):
                q = c["q"][b, t, h // 3]
                want[b, t, h] = a ** (t + 1) * (q @ c["S0"][b, h])
                for s in range(t + 1):
                    want[b, t, h] += a ** (t - s) * (q @ c["k"][b, s, h // 2]) * c["v"][b, s, h]
    assert np.allclose(out, 0.7 * want)
    short, held = oracle.linear_attention(c["q"][1:, :3], c["k"][1:, :3], c["v"][1:, :3], c["rate"], 0.7, c["S0"][1:])
    assert np.allclose(out[1, :3], short[0]) and np.allclose(last[1], held[0]) and not out[1, 3:].any()


@pytest.mark.parametrize("name", ["q", "k", "v", "S0"])
def test_attention_gradients_are_differences(name):
    rng = np.random.default_rng(2)
    c = attention_inputs(rng)
    d, e = rng.standard_normal((2, 5, 6, 4)), rng.standard_normal((2, 6, 3, 4))
    g = oracle.linear_attention_bwd(c["q"], c["k"], c["v"], c["rate"], 0.7, d, c["S0"], c["seq_lens"], e)
    m = oracle.linear_attention_bwd(c["q"], c["k"], c["v"], c["rate"], 0.7, d, c["S0"], c["seq_lens"], e, magnitude=True)

    def f(x):
        a = dict(c, **{name: x})
        out, last = oracle.linear_attention(a["q"], a["k"], a["v"], a["rate"], 0.7, a["S0"], a["seq_lens"])
        return np.sum(d * out) + np.sum(e * last)

    agree(f, c[name], g["d" + name], rng)
    assert np.all(m["d" + name] >= np.abs(g["d" + name]) - 1e-12)


def test_logprobs_of_equal_logits_and_of_masked_ones():
    x = np.array([[2.0, 2.0, -np.inf, 2.0, 2.0], [-np.inf] * 5, [0.0, np.nan, 1.0, 0.0, 0.0], [0.0, np.inf, 1.0, 0.0, 0.0]])
    o = oracle.token_logprobs(x, np.array([3, 1, 0, 2]), top=4)
    assert np.allclose(o["logprobs"][0], -np.log(4)) and np.allclose(o["entropy"][0], np.log(4))
    assert o["logprobs"][1] == -np.inf and o["entropy"][1] == 0 and np.isnan(o["logprobs"][2:]).all()
    assert np.isnan(o["entropy"][2:]).all()
    assert list(o["top_tokens"][0]) == [0, 1, 3, 4] and list(o["top_tokens"][1]) == [-1] * 4
    assert list(o["top_tokens"][2]) == [2, 0, 3, 4]
    assert oracle.token_logprobs(x[:1], np.array([5]))["logprobs"][0] == 0
    assert oracle.token_logprobs(x[:1], np.array([-1]))["logprobs"][0] == 0


def test_logprob_gradients_are_differences():
    rng = np.random.default_rng(3)
    x, t = rng.standard_normal((4, 9)), np.array([0, 8, 3, -1])
    g, h = rng.standard_normal(4), rng.standard_normal(4)

    def f(a):
        o = oracle.token_logprobs(a, t)
        return np.sum(g * o["logprobs"]) + np.sum(h * o["entropy"])

    d, m = oracle.token_logprobs_bwd(x, t, g, h)
    agree(f, x, d, rng)
    assert np.all(m >= np.abs(d) - 1e-12)
    x[1, 2:5] = -np.inf
    d, _ = oracle.token_logprobs_bwd(x, t, g, h)
    assert not d[1, 2:5].any() and abs(d[1].sum()) < 1e-12
