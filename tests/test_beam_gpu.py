"""GPU tests of beam search's selection and state reordering against the fp64 definitions.

A selected score is the definition's sum rounded once to fp32 (u = 2^-24 of it) plus the error of the
normaliser: a sum of exponentials, each off by (|logit - max| + 4) u of itself (those far below the
maximum weigh nothing: |logit - max| e^(logit - max) < 0.4), added up over at most V / 64 + 16 steps.
Parents and tokens are equal to the definition's wherever its score stands further from its neighbours
than twice that, or equals them with its order defined: within a beam, and between beams whose logits and
scores are copies (their normalisers are then the same sums in the same order; those of a row and its
reverse agree to rounding alone)."""
import numpy as np
import pytest

import oracle
from synth import round_to_bf16
from tests.gpu_helpers import dev
from tests.test_gated_gpu import mss  # noqa: F401

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def run_and_check(mss, logits, scores, dtype="f32", k=None, finished=None, end=None, off=0, mixed=False):  # noqa: F811
    import torch
    x = dev(logits, dtype)
    if off:
        flat = torch.empty(x.numel() + off, dtype=x.dtype, device="cuda")
        flat[off:].copy_(x.reshape(-1))
        x = flat[off:].view(x.shape)
    fin = None if finished is None else torch.from_numpy(np.ascontiguousarray(finished, np.int32)).cuda()
    got = mss.beam_select(x, dev(scores), finished=fin, end_token=end, k=k)
    ref = oracle.beam_select(logits, scores, k=k, finished=finished, end_token=end)
    s, p, v = (t.cpu().numpy() for t in got[:3])
    rs = ref[0]
    assert s.shape == rs.shape
    np.testing.assert_array_equal(np.isfinite(s), np.isfinite(rs))
    ok = np.isfinite(rs)
    tol = (np.abs(np.where(ok, rs, 0)) + logits.shape[2] / 64 + 24) * U
    assert np.all(np.abs(np.where(ok, s - np.where(ok, rs, 0), 0)) <= tol)
    r0 = np.where(ok, rs, -1e300)
    gap = np.full(rs.shape, np.inf)
    d = np.abs(np.diff(r0, axis=1))
    par = ref[1]
    for b in range(par.shape[0]):
        for j in np.flatnonzero(d[b] == 0):
            one, two = par[b, j], par[b, j + 1]
            if one == two or (scores[b, one] == scores[b, two] and np.array_equal(logits[b, one], logits[b, two])):
                d[b, j] = np.inf
    gap[:, 1:] = np.minimum(gap[:, 1:], d)
    gap[:, :-1] = np.minimum(gap[:, :-1], d)
    sure = gap > 2 * tol.max()
    assert mixed or sure.mean() > 0.9  # the inputs leave hardly anything open
    np.testing.assert_array_equal(p[sure], ref[1][sure])
    np.testing.assert_array_equal(v[sure], ref[2][sure])
    if finished is not None:
        np.testing.assert_array_equal(got[3].cpu().numpy()[sure], ref[3][sure])
    return got


def make(B, N, V, dtype, seed, scale=2.5):
    rng = np.random.default_rng(seed)
    x = (scale * rng.standard_normal((B, N, V))).astype(np.float32)
    return (round_to_bf16(x) if dtype == "bf16" else x), (-rng.uniform(1, 20, (B, N))).astype(np.float32), rng


@pytest.mark.parametrize("B,N,V,k,dtype", [
    (1, 1, 1, 1, "f32"), (2, 2, 1, 2, "bf16"), (2, 3, 5, 3, "f32"), (1, 4, 7, 8, "bf16"), (3, 4, 511, 4, "f32"),
    (2, 4, 512, 4, "bf16"), (2, 5, 513, 10, "f32"), (1, 4, 32768, 4, "bf16"), (4, 8, 50001, 16, "bf16"),
    (2, 3, 128007, 3, "f32"), (1, 1, 65536, 64, "f32"), (1, 64, 1000, 64, "bf16"), (70, 2, 3000, 2, "f32"),
    (1, 2, 40, 64, "f32"), (300, 16, 1001, 16, "bf16")])
def test_selection(mss, B, N, V, k, dtype):  # noqa: F811
    x, s, rng = make(B, N, V, dtype, B + N + V + k)
    run_and_check(mss, x, s, dtype, k)
    fin = (rng.random((B, N)) < 0.4).astype(np.int32) * 3
    run_and_check(mss, x, s, dtype, k, finished=fin, end=V // 2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [4096, 4099])
def test_rows_that_start_anywhere(mss, dtype, V):  # noqa: F811
    x, s, _ = make(2, 3, V, dtype, V)
    for off in (1, 3):
        run_and_check(mss, x, s, dtype, off=off)


def test_ties_go_by_beam_then_logit_then_token(mss):  # noqa: F811
    """Logits of five values (hundreds of equal ones in every slice), beams that are copies of each
    other with the same score, rising and falling rows."""
    rng = np.random.default_rng(3)
    x = rng.integers(0, 5, (2, 6, 20000)).astype(np.float32)
    x[:, 3] = x[:, 1]
    x[1, 4] = np.sort(x[1, 4])
    x[1, 5] = np.sort(x[1, 5])[::-1]
    x[0, 5] = 2.0
    s = np.array([[-3, -1, -7, -1, -2, -1]] * 2, np.float32)
    run_and_check(mss, x, s, "f32", 24)
    run_and_check(mss, x, s, "bf16", 24)
    zeros = np.zeros((1, 3, 2000), np.float32)  # zeros of both signs are equal
    zeros[:, :, ::3] = -0.0
    run_and_check(mss, zeros, np.array([[-1, -0.0, 0.0]], np.float32), "f32", 40)
    run_and_check(mss, zeros, np.array([[-1, -0.0, 0.0]], np.float32), "bf16", 40)
    up = np.arange(30000, dtype=np.float32)[None, None] * 1e-3  # every tile beats the list
    x = np.concatenate([up, up[..., ::-1]], 1)
    got = run_and_check(mss, x, np.zeros((1, 2), np.float32), "f32", 32, mixed=True)
    pairs = list(zip(got[1][0].tolist(), got[2][0].tolist()))
    for beam, tokens in ((0, range(29999, 29983, -1)), (1, range(16))):  # each beam's own order
        assert [v for p, v in pairs if p == beam] == list(tokens)


def test_masked_rows_and_unused_beams(mss):  # noqa: F811
    x, s, _ = make(4, 4, 3000, "f32", 5)
    x[0, 1] = -np.inf                      # nothing left in a beam
    x[1] = -np.inf                         # nothing left in a request
    x[2, 0, :2990] = -np.inf               # ten left
    x[2, 1:] = -np.inf
    x[3, 0, 7] = np.nan                    # a masked NaN
    x[3, 1, :] = np.nan
    x[3, 2, 9] = np.inf                    # a row without a softmax
    s[0, 2:] = -np.inf                     # beams not used yet
    got = run_and_check(mss, x, s, "f32", 16)
    assert (got[0][1] == -np.inf).all() and not got[1][1].any() and not got[2][1].any()
    s[3, 3] = np.nan
    run_and_check(mss, x, s, "f32", 16)
    # masks of the type's lowest value, and scores of it for unused beams: finite, and last
    low = np.float32(np.finfo(np.float32).min)
    x, s, _ = make(2, 3, 500, "f32", 6)
    x[:, :, 3:] = low
    s[:, 1:] = low
    got = mss.beam_select(dev(x), dev(s), k=3)
    want = oracle.beam_select(x, s, k=3)
    assert got[1].tolist() == want[1].tolist() == [[0, 0, 0]] * 2 and got[2].tolist() == want[2].tolist()
    s[:] = 0
    fin = np.array([[1, 1, 1], [0, 1, 0]], np.int32)  # a request whose beams are all at their end
    x, _, _ = make(2, 3, 500, "f32", 7)
    run_and_check(mss, x, s - np.array([[1, 2, 3.5]], np.float32), "f32", 6, finished=fin, end=499)


def test_in_place_and_again(mss):  # noqa: F811
    import torch
    x, s, rng = make(5, 8, 9001, "f32", 11)
    fin = torch.from_numpy((rng.random((5, 8)) < 0.3).astype(np.int32)).cuda()
    xd, sd = dev(x), dev(s)
    a = mss.beam_select(xd, sd, finished=fin, end_token=4)
    b = mss.beam_select(xd, sd, finished=fin, end_token=4)
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    c = mss.beam_select(xd, sd, finished=fin, end_token=4, next_scores=sd, next_finished=fin)
    assert c[0] is sd and c[3] is fin and all(torch.equal(u, v) for u, v in zip(a, c))


def test_selection_past_2_to_the_31_logits(mss):  # noqa: F811
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty((300, 56, 131071), dtype=torch.bfloat16, device="cuda").normal_(generator=g)  # 2.2e9
    s = -torch.rand((300, 56), generator=g, device="cuda") * 9
    a = mss.beam_select(x, s, k=8)
    b = mss.beam_select(x[-1:].contiguous(), s[-1:].contiguous(), k=8)
    # the single request is cut into other slices: its normalisers may differ in the last bits
    assert float((a[0][-1:] - b[0]).abs().max()) <= (20 + 2 * (131071 / 64 + 24)) * U
    assert torch.equal(a[1][-1:], b[1]) and torch.equal(a[2][-1:], b[2])


REORDER = [(1, 1, [(3,)]), (2, 4, [(5, 16), (5, 3), (7,), ()]), (3, 3, [(33, 16), (33, 5)]), (2, 8, [(640, 16), (640, 3)]),
           (1, 16, [(257, 4)]), (2, 17, [(100, 8), (9,)]), (1, 64, [(130, 16), (3, 3)]), (5, 2, [(1,)] * 40),
           (2, 4, [(0,), (6, 0), (8,)])]


@pytest.mark.parametrize("B,N,shapes", REORDER)
def test_reorder(mss, B, N, shapes):  # noqa: F811
    import torch
    rng = np.random.default_rng(B + N)
    for parents in (rng.integers(0, N, (B, N)), np.tile(np.arange(N), (B, 1)), np.zeros((B, N), int),
                    np.tile(np.arange(N)[::-1], (B, 1)), rng.integers(-3, N + 3, (B, N))):
        par = torch.from_numpy(np.ascontiguousarray(parents, np.int32)).cuda()
        st, want = [], []
        for j, shape in enumerate(shapes):
            a = rng.standard_normal((B * N, *shape)).astype(np.float32)
            t = torch.from_numpy(a).cuda()
            t = (t, t.to(torch.bfloat16), (t * 1000).to(torch.int32))[j % 3]
            if j % 2 and t.numel():  # off a 16-byte boundary
                flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
                flat[1:].copy_(t.reshape(-1))
                t = flat[1:].view(t.shape)
            st.append(t)
            w = t.cpu()
            want.append(torch.from_numpy(oracle.beam_reorder(np.arange(B * N), parents)))
            want[-1] = w[want[-1]]
        guard = torch.full((64,), 7.0, device="cuda")
        got = mss.beam_reorder(st, par)
        assert got is st and float(guard.sum()) == 448
        for a, b in zip(st, want):
            assert torch.equal(a.cpu(), b)


def test_reorder_past_2_to_the_31_bytes(mss):  # noqa: F811
    import torch
    st = torch.arange(8, device="cuda", dtype=torch.int32)[:, None].expand(8, 150_000_001).contiguous()
    mss.beam_reorder([st], torch.tensor([[3, 2, 1, 1], [0, 0, 2, 0]], dtype=torch.int32, device="cuda"))
    want = torch.tensor([3, 2, 1, 1, 4, 4, 6, 4], dtype=torch.int32, device="cuda")
    assert torch.equal(st[:, 0], want) and torch.equal(st[:, -1], want)
    assert bool((st == want[:, None]).all())


def test_captured_step_replayed(mss):  # noqa: F811
    """BeamSearchStep captured with no call before on its own stream: every replay, on new logits,
    equals the eager calls bit for bit."""
    import torch
    x, s, _ = make(3, 4, 5000, "bf16", 21)
    xd, sd = dev(x, "bf16"), dev(s)
    fin = torch.zeros((3, 4), dtype=torch.int32, device="cuda")
    states = [torch.randn((12, 50, 16), device="cuda"), torch.randn((12, 50, 3), device="cuda").to(torch.bfloat16)]
    stream = torch.cuda.Stream()
    step = mss.BeamSearchStep(xd, sd, states, finished=fin, end_token=17, stream=stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    es, ef, est = sd.clone(), fin.clone(), [t.clone() for t in states]
    for rep in range(4):
        nx, _, _ = make(3, 4, 5000, "bf16", 30 + rep)
        nx[0, 0, 17] = 40.0  # somebody reaches the end
        xd.copy_(dev(nx, "bf16"))
        _, p, v, _ = mss.beam_select(xd, es, finished=ef, end_token=17, next_scores=es, next_finished=ef)
        mss.beam_reorder(est, p)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(step.parents, p) and torch.equal(step.tokens, v), rep
        assert torch.equal(sd, es) and torch.equal(fin, ef), rep
        assert all(torch.equal(a, b) for a, b in zip(states, est)), rep
    assert fin.any()
