"""GPU tests of token log probabilities, entropies, alternatives and the gradient to the logits against the fp64 definition.

Tolerances, with u = 2^-24 and d = x - m <= 0, |d| <= 40 for these inputs where e^d counts (e^d |d| falls beyond):
  - e^d: d has a rounding, d log2 e two more, exp2 two u: (3 |d| + 3) u of a term; terms are weighted by themselves, and
    the sum over p of |d| is below 16 here: 51 u; a lane adds a tile's 8 terms, then its tiles n = vocab / 4096 + 1, and rescales
    when its m rises: (8 + 2 n) u.  So log s is (60 + 2 n) u off, the log probability that and a rounding of itself.
  - t / s: t's terms carry |d| more; (60 + 2 n + 3) u of |t| / s and as much for s.
  - a gradient's p: (3 |d| + 3 + 60 + 2 n) u with |d| <= 40: (183 + 2 n) u of the terms' magnitudes; entropy - log s the same.
A bf16 gradient adds half a step, 2^-8 of its value."""
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


def inputs(R, V, dtype, seed=0, masked=False, scale=2.5):
    rng = np.random.default_rng(9000 + seed)
    x = (rng.standard_normal((R, V)) * scale).astype(np.float32)
    t = rng.integers(0, V, R).astype(np.int32)
    if masked:
        x[rng.random((R, V)) < 0.4] = -np.inf
    x = round_to_bf16(x) if dtype == "bf16" else x
    return dict(x=x, t=t, g=rng.standard_normal(R).astype(np.float32), h=rng.standard_normal(R).astype(np.float32), dtype=dtype)


def tokens(t):
    import torch
    return torch.from_numpy(np.asarray(t, dtype=np.int32)).cuda()


def same_kind(g, ref):
    assert np.array_equal(np.isnan(g), np.isnan(ref)) and np.array_equal(np.isinf(g), np.isinf(ref))
    assert np.array_equal(g[np.isinf(ref)], ref[np.isinf(ref)])


def close(got, ref, lim, what):
    g = host64(got).reshape(ref.shape)
    same_kind(g, ref)
    f = np.isfinite(ref)
    bad = np.abs(g - ref)[f] > np.broadcast_to(lim, ref.shape)[f]
    assert not bad.any(), (what, int(bad.sum()), float(np.max((np.abs(g - ref) / lim)[f])))


def check(mss, c, top=0, entropy=True):
    V, n = c["x"].shape[1], c["x"].shape[1] / 4096 + 1
    x, t = dev(c["x"], c["dtype"]), tokens(c["t"])
    o = oracle.token_logprobs(c["x"], c["t"], top)
    base = (62 + 2 * n) * U
    got = mss.token_logprobs(x, t, top=top)
    close(got[0], o["logprobs"], base + 2 * U * np.abs(np.nan_to_num(o["logprobs"], neginf=0)), "logprobs")
    close(got[1], o["entropy"], 2 * base * (1 + 16), "entropy")
    if top:
        assert np.array_equal(got[3].cpu().numpy(), o["top_tokens"])
        close(got[2], o["top_logprobs"], base + 2 * U * np.abs(np.nan_to_num(o["top_logprobs"], neginf=0)), "top_logprobs")
    lp, en, saved = mss.token_logprobs_save(x, t)
    if not top:
        assert np.array_equal(host64(lp), host64(got[0]), equal_nan=True)
    h = c["h"] if entropy else None
    d = mss.token_logprobs_bwd(x, t, saved, dev(c["g"]), dev(h))
    ref, M = oracle.token_logprobs_bwd(c["x"], c["t"], c["g"], h)
    half = 2.0 ** -8 if c["dtype"] == "bf16" else 0.0
    with np.errstate(invalid="ignore"):
        lim = (190 + 2 * n) * U * (M + np.abs(c["h"])[:, None] * o["p"]) + half * np.abs(ref) + 1e-37
    close(d, ref, lim, "dlogits")
    return x, t, saved, d


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,V", [(1, 1), (3, 2), (5, 7), (2, 64), (4, 511), (4, 512), (3, 513), (2, 4096), (7, 5003), (1, 50277),
                                 (3, 32768), (700, 1000), (2, 131072)])
def test_sizes(mss, R, V, dtype):
    check(mss, inputs(R, V, dtype, R + V), top=min(V, 20))
    check(mss, inputs(R, V, dtype, R + V + 1, masked=True), entropy=False)


@pytest.mark.parametrize("top", [1, 2, 3, 17, 63, 64])
def test_alternatives(mss, top):
    for V in (40, 640, 9000, 40000):
        check(mss, inputs(3, V, "bf16", V + top), top=top)        # bf16 logits have many ties
        check(mss, inputs(3, V, "f32", V + top, masked=True), top=top)


def test_ties_go_to_the_lowest_token(mss):
    x = np.zeros((4, 30000), dtype=np.float32)
    x[1, 29990:] = 1.0
    x[2, ::3] = -0.0
    x[3] = -np.inf
    x[3, [7, 12345, 29999]] = 2.0
    c = dict(x=x, t=np.array([0, 29999, 5, 7], dtype=np.int32), g=np.ones(4, np.float32), h=np.ones(4, np.float32), dtype="f32")
    check(mss, c, top=12)


def test_masked_rows_missing_tokens_infinities_and_nan(mss):
    import torch
    rng = np.random.default_rng(1)
    x = rng.standard_normal((8, 3000)).astype(np.float32)
    x[0] = -np.inf                       # nothing left
    x[1] = -np.inf
    x[1, 2999] = -50.0                   # one left
    x[2, 40] = np.nan
    x[3, 50] = np.inf
    x[4] = -3.4e38                       # the type's lowest value as a mask, one allowed
    x[4, 9] = 1.0
    x[5] = np.nan
    t = np.array([4, 2999, 7, 8, 9, 0, -1, 3000], dtype=np.int32)
    c = dict(x=x, t=t, g=np.ones(8, np.float32), h=np.full(8, 0.5, np.float32), dtype="f32")
    xd, td = dev(x), tokens(t)
    o = oracle.token_logprobs(x, t, 5)
    lp, en, tl, tt = mss.token_logprobs(xd, td, top=5)
    close(lp, o["logprobs"], 70 * U * (1 + np.abs(np.nan_to_num(o["logprobs"], neginf=0))), "logprobs")
    close(en, o["entropy"], 2400 * U, "entropy")
    assert np.array_equal(tt.cpu().numpy(), o["top_tokens"])
    same_kind(host64(tl), o["top_logprobs"])
    assert list(tt[0].cpu()) == [-1] * 5 and list(tt[1].cpu()) == [2999] + [-1] * 4
    assert float(lp[0]) == -np.inf and float(lp[1]) == 0 and float(lp[6]) == 0 and float(lp[7]) == 0
    _, _, saved = mss.token_logprobs_save(xd, td)
    d = mss.token_logprobs_bwd(xd, td, saved, dev(c["g"]), dev(c["h"]))
    assert not d[0].any() and not d[1].any() and torch.isnan(d[2]).all() and torch.isnan(d[5]).all()
    ref, M = oracle.token_logprobs_bwd(x, t, c["g"], c["h"])
    rows = [0, 1, 4, 6, 7]
    close(d[rows], ref[rows], (260 * U * (M + 1e-3) + 1e-37)[rows], "dlogits")


def test_in_place_shapes_and_unaligned_rows(mss):
    import torch
    c = inputs(6, 1003, "bf16", 3)
    x, t, saved, d = check(mss, c)
    y = x.clone()
    before = y._version
    same = mss.token_logprobs_bwd(y, t, saved, dev(c["g"]), dev(c["h"]), dlogits=y)
    assert same is y and torch.equal(y, d) and y._version > before
    lp3, en3, tl3, tt3 = mss.token_logprobs(x.view(2, 3, 1003), t.view(2, 3), top=4)
    lp, en, tl, tt = mss.token_logprobs(x, t, top=4)
    assert torch.equal(lp3.flatten(), lp) and torch.equal(tt3.flatten(0, 1), tt) and tl3.shape == (2, 3, 4)
    big = torch.full((6 * 1003 + 9,), 9.0, dtype=torch.bfloat16, device="cuda")
    view = big[1:1 + 6 * 1003].view(6, 1003)
    view.copy_(x)
    assert torch.equal(mss.token_logprobs(view, t)[0], lp)
    mss.token_logprobs_bwd(view, t, saved, dev(c["g"]), dev(c["h"]), dlogits=view)
    assert torch.equal(view, d) and float(big[0]) == 9.0 and bool((big[-8:] == 9.0).all())
    none = torch.empty(0, 50, device="cuda")
    assert mss.token_logprobs(none, tokens([]), top=3)[3].shape == (0, 3)


def test_rows_past_31_bits_of_logits(mss):
    import torch
    R, V = 16800, 128007
    rows = [0, 1, 8388, 16776, R - 1]
    c = inputs(len(rows), V, "bf16", 5)
    x = torch.zeros(R, V, dtype=torch.bfloat16, device="cuda")
    x[rows] = dev(c["x"], "bf16")
    t = torch.zeros(R, dtype=torch.int32, device="cuda")
    t[rows] = tokens(c["t"])
    g, h = torch.zeros(R, device="cuda"), torch.zeros(R, device="cuda")
    g[rows], h[rows] = dev(c["g"]), dev(c["h"])
    lp, en, tl, tt = mss.token_logprobs(x, t, top=3)
    o, n = oracle.token_logprobs(c["x"], c["t"], 3), V / 4096 + 1
    close(lp[rows], o["logprobs"], (62 + 2 * n) * U + 2 * U * np.abs(o["logprobs"]), "logprobs")
    assert np.array_equal(tt[rows].cpu().numpy(), o["top_tokens"])
    _, _, saved = mss.token_logprobs_save(x, t)
    mss.token_logprobs_bwd(x, t, saved, g, h, dlogits=x)
    ref, M = oracle.token_logprobs_bwd(c["x"], c["t"], c["g"], c["h"])
    close(x[rows], ref, (190 + 2 * n) * U * (M + np.abs(c["h"])[:, None] * o["p"]) + 2.0 ** -8 * np.abs(ref) + 1e-37, "dlogits")


def test_graph_side_stream_and_autograd(mss):
    import torch
    c = inputs(9, 20001, "f32", 7)
    x, t, g, h = dev(c["x"]), tokens(c["t"]), dev(c["g"]), dev(c["h"])

    def step():
        lp, en, saved = mss.token_logprobs_save(x, t)
        return [lp, en, mss.token_logprobs_bwd(x, t, saved, g, h), *mss.token_logprobs(x, t, top=6)]

    want = step()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        got = step()
    for _ in range(3):
        [a.zero_() for a in got]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(step(), want))
    leaf = x.clone().requires_grad_()
    lp, en = mss.TokenLogprobsFunction.apply(leaf, t)
    torch.autograd.backward([lp, en], [g, h])
    assert torch.equal(leaf.grad, want[2])
    leaf2 = x.clone().requires_grad_()
    mss.TokenLogprobsFunction.apply(leaf2, t)[0].mean().backward()  # a loss without the entropy
    mean = torch.full_like(g, 1 / 9)
    assert torch.equal(leaf2.grad, mss.token_logprobs_bwd(x, t, mss.token_logprobs_save(x, t)[2], mean, torch.zeros_like(g)))


def test_alternatives_of_many_equal_logits_and_at_the_ends(mss):
    """Rows whose lanes all hold the k-th greatest logit, and whose alternatives are their first and last tokens."""
    rng = np.random.default_rng(31)
    for V in (9, 517, 4099, 20001):
        x = np.zeros((5, V), dtype=np.float32)
        x[1] = rng.integers(0, 3, V)
        x[2, -5:] = np.arange(5) + 1.0
        x[2, :3] = 9.0
        x[3] = np.arange(V, dtype=np.float32) / V
        x[4] = -np.arange(V, dtype=np.float32) / V
        c = dict(x=round_to_bf16(x), t=np.array([0, 1, V - 1, V // 2, 0], dtype=np.int32), g=np.ones(5, np.float32),
                 h=np.ones(5, np.float32), dtype="bf16")
        for top in (1, 7, 64):
            check(mss, c, top=min(top, V))


def test_alternatives_of_long_rows_in_one_block(mss):
    """More rows than are cut, of more tiles to a wave than are read again at once; in distinct and in equal logits."""
    import torch
    R, V, k = 1030, 140001, 20
    x = torch.randn(R, V, device="cuda")
    t = torch.zeros(R, dtype=torch.int32, device="cuda")
    _, _, tl, tt = mss.token_logprobs(x, t, top=k)
    for rows in torch.arange(R, device="cuda").split(103):
        want = x[rows].topk(k, -1)[0]
        assert torch.equal(x[rows].gather(-1, tt[rows].long()), want)
        s = tt[rows].sort(-1)[0]
        assert bool((s[:, 1:] > s[:, :-1]).all())
    x.zero_()
    tt = mss.token_logprobs(x, t, top=k)[3]
    assert torch.equal(tt, torch.arange(k, dtype=torch.int32, device="cuda").expand(R, k))


def test_more_rows_than_blocks(mss):
    import torch
    R, V = (1 << 22) + 7, 3
    x = torch.randn(R, V, device="cuda")
    t = torch.randint(0, V, (R,), device="cuda", dtype=torch.int32)
    lp, en, tl, tt = mss.token_logprobs(x, t, top=2)
    p = torch.log_softmax(x.double(), -1)
    want = p.gather(-1, t.long()[:, None])[:, 0]
    assert bool(((lp - want).abs() <= 64 * U + 2 * U * want.abs()).all())
    assert bool(((en + (p.exp() * p).sum(-1)).abs() <= 2 * 64 * U * 17).all())
    assert torch.equal(x.gather(-1, tt.long()), x.topk(2, -1)[0])
    _, _, saved = mss.token_logprobs_save(x, t)
    d = mss.token_logprobs_bwd(x, t, saved, torch.ones(R, device="cuda"))
    want = torch.nn.functional.one_hot(t.long(), V) - p.exp()
    assert bool(((d - want).abs() <= 192 * U * (1 + p.exp())).all())


@pytest.mark.parametrize("dtype,V", [("bf16", 50280), ("bf16", 50281), ("f32", 25004)])
def test_gradients_larger_than_the_cache(mss, dtype, V):
    """Rows that are and are not whole vectors, of more logits than are kept for the next reader; also in place."""
    import torch
    R = 1400
    x = (torch.randn(R, V, device="cuda") * 2.5).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    assert x.numel() * x.element_size() > 1 << 27
    rows = [0, 1, 701, R - 1]
    t = torch.randint(0, V, (R,), device="cuda", dtype=torch.int32)
    g, h = torch.randn(R, device="cuda"), torch.randn(R, device="cuda")
    _, _, saved = mss.token_logprobs_save(x, t)
    d = mss.token_logprobs_bwd(x, t, saved, g, h)
    xr, n = host64(x[rows]).astype(np.float32), V / 2048 + 1
    ref, M = oracle.token_logprobs_bwd(xr, t[rows].cpu().numpy(), g[rows].cpu().numpy(), h[rows].cpu().numpy())
    p = np.exp(xr - xr.max(-1, keepdims=True), dtype=np.float64)
    p /= p.sum(-1, keepdims=True)
    lim = (190 + 2 * n) * U * (M + np.abs(h[rows].cpu().numpy())[:, None] * p) + (2.0 ** -8 if dtype == "bf16" else 0.0) * np.abs(ref)
    close(d[rows], ref, lim + 1e-37, "dlogits")
    mss.token_logprobs_bwd(x, t, saved, g, h, dlogits=x)
    assert torch.equal(x, d)
