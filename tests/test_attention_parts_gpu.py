"""GPU tests of linear attention in bf16 where large terms of an output cancel: states and scores keep fp32's precision on
their way through the matrix cores, so that only the result is rounded to bf16.

Tolerances, u = 2^-24, rate 0 and scale 1 (every decay is 1 exactly), M the sum of the terms' magnitudes:
  - a state met by queries that are +1 once, -1 once and otherwise 0: three bf16 parts leave 2^-27 of a value, the products
    are exact, the six of them that are not 0 take five additions: 8 u M holds it.
  - scores of queries and keys with five nonzero columns: exact products, four additions; three parts; an output that adds
    two scores, six products and five additions: 12 u M holds it.
  - a bf16 result adds half a step, 2^-8 of its value.
Two parts of a value would leave up to 2^-18 of it: 64 u."""
import numpy as np
import pytest

import oracle
from synth import round_to_bf16
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


def close(got, ref, M, n, what):
    g = host64(got)
    lim = n * U * M + 2.0 ** -8 * np.abs(ref) + 1e-37
    assert g.shape == ref.shape and np.all(np.isfinite(g)), what
    assert np.all(np.abs(g - ref) <= lim), (what, float(np.max(np.abs(g - ref) / lim)))


def differences(rng, *shape):
    """Rows with one +1, one -1 and zeros."""
    x = np.zeros(shape, dtype=np.float32)
    rows = x.reshape(-1, shape[-1])
    for r in rows:
        i, j = rng.choice(shape[-1], 2, replace=False)
        r[i], r[j] = 1.0, -1.0
    return x


@pytest.mark.parametrize("K,V", [(32, 32), (128, 64), (64, 128), (128, 128)])
def test_states(mss, K, V):
    B, L, H = 2, 70, 2
    rng = np.random.default_rng(K + V)
    rate, zero = np.zeros(H, dtype=np.float32), lambda *s: np.zeros(s, dtype=np.float32)  # noqa: E731
    near = rng.standard_normal((B, H, 1, 1)) + 2.0 ** -12 * rng.standard_normal((B, H, K, V))
    S = near.astype(np.float32)
    q, k, v, d = differences(rng, B, L, H, K), differences(rng, B, L, H, K), differences(rng, B, L, H, V), differences(rng, B, L, H, V)
    kz, vz = zero(B, L, H, K), zero(B, L, H, V)
    run = lambda a: [dev(t, "bf16") for t in a]  # noqa: E731

    out, last = mss.linear_attention_fwd(*run((q, kz, vz)), dev(rate), scale=1.0, initial_state=dev(S))
    ref = np.einsum("blhk,bhkv->blhv", q.astype(np.float64), S)
    close(out, ref, np.einsum("blhk,bhkv->blhv", np.abs(q), np.abs(S)), 8, "out")
    assert np.array_equal(last.cpu().numpy(), S)
    g = mss.linear_attention_bwd(*run((kz, kz, vz)), dev(rate), dev(d, "bf16"), scale=1.0, initial_state=dev(S))
    ref = np.einsum("blhv,bhkv->blhk", d.astype(np.float64), S)
    close(g["dq"], ref, np.einsum("blhv,bhkv->blhk", np.abs(d), np.abs(S)), 8, "dq")
    g = mss.linear_attention_bwd(*run((kz, k, v)), dev(rate), dev(vz, "bf16"), scale=1.0, dlast_state=dev(S))
    ref = np.einsum("blhv,bhkv->blhk", v.astype(np.float64), S)
    close(g["dk"], ref, np.einsum("blhv,bhkv->blhk", np.abs(v), np.abs(S)), 8, "dk")
    ref = np.einsum("blhk,bhkv->blhv", k.astype(np.float64), S)
    close(g["dv"], ref, np.einsum("blhk,bhkv->blhv", np.abs(k), np.abs(S)), 8, "dv")


def few(rng, L, D):
    """Rows with four columns of [1, 2) and 2^-8 in a fifth."""
    x = np.zeros((L, D), dtype=np.float32)
    x[:, :4] = round_to_bf16(rng.uniform(1.0, 2.0, (L, 4)).astype(np.float32))
    x[:, 4] = 2.0 ** -8
    return x


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("K,V", [(32, 32), (128, 64), (64, 128), (128, 128)])
def test_scores(mss, K, V, shared):
    """Two keys that differ in the fifth column alone, with values of opposite signs: an output is the difference of two
    scores of about 8, 2^-11.  Walked forwards for out and dq, backwards for dk and dv."""
    L, H = 32, 3
    rng = np.random.default_rng(100 + K + V)
    rate, heads = np.zeros(H, dtype=np.float32), 1 if shared else H

    def many(n, D):
        return np.stack([few(rng, L, D) for _ in range(n)], 1)[None]

    def two(n, D, at):  # equal rows at two steps but for the fifth column, zeros at the others
        x = np.zeros((1, L, n, D), dtype=np.float32)
        x[:, at[0]] = x[:, at[1]] = few(rng, n, D)
        x[:, at[0], :, 4], x[:, at[1], :, 4] = 0.0, 2.0 ** -3
        return x

    def signs(n, D, at):
        x = np.zeros((1, L, n, D), dtype=np.float32)
        x[:, at[0]] = rng.choice([-1.0, 1.0], (n, D))
        x[:, at[1]] = -x[:, at[0]]
        return x

    def check(q, k, v, d, names):
        t = [dev(x, "bf16") for x in (q, k, v)]
        args = (q, k, v, rate, 1.0)
        ref, M = {"out": oracle.linear_attention(*args)[0]}, {"out": oracle.linear_attention(*args, magnitude=True)[0]}
        ref.update(oracle.linear_attention_bwd(*args, d))
        M.update(oracle.linear_attention_bwd(*args, d, magnitude=True))
        got = {"out": mss.linear_attention_fwd(*t, dev(rate), scale=1.0)[0]}
        got.update(mss.linear_attention_bwd(*t, dev(rate), dev(d, "bf16"), scale=1.0))
        for n in names:  # (a head that several share adds their terms: two additions more)
            close(got[n], ref[n], M[n], 16, n)

    first, last = (0, 1), (L - 1, L - 2)
    dout = np.zeros((1, L, H, V), dtype=np.float32)
    check(many(heads, K), two(heads, K, first), signs(heads, V, first), dout, ["out"])
    check(many(heads, K), signs(heads, K, first), two(heads, V, first), many(H, V), ["dq"])
    check(two(heads, K, last), many(heads, K), many(heads, V), signs(H, V, last), ["dv"])
    check(signs(heads, K, last), many(heads, K), many(heads, V), two(H, V, last), ["dk"])
