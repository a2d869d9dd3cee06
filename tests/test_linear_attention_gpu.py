"""GPU tests of linear attention (sequences, gradients, one token) against the fp64 definition, which goes step by step.

Tolerances, with u = 2^-24 and M the same sums with every term's magnitude:
  - a power l^n: its exponent rate n log2 e has two roundings, exp2 two u more, and it is formed of at most two powers and
    a factor: (4 e + 10) u with e = rate n <= 64 rate_max; a term with a larger n has passed through the state.
  - the state over c chunks: S + S expm1(-rate C), 4 u and a rounding each: 6 c u.
  - sums: a score adds up to key_dim products, an output those of the state and the chunk, one rounding each at most: 3 * 192 u
    over the three products a term passes.
  - parts: bf16 inputs: scores and states 2^-17 each; fp32 inputs: each of three products 4 * 2^-24.
So C = (4 * 64 rate_max + 10 + 6 c + 576 + 12) u, + 2^-16 for bf16, of M; a bf16 result adds half a step, 2^-8 of its
value.  Shared heads add H more u."""
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


def inputs(B, L, H, K, V, dtype, heads=None, lens=False, state=False, seed=0, rate=(0.0005, 0.03)):
    rng = np.random.default_rng(8000 + seed)
    heads = heads or (H, H, H)

    def draw(*s):
        a = rng.standard_normal(s).astype(np.float32)
        return round_to_bf16(a) if dtype == "bf16" else a

    c = dict(q=draw(B, L, heads[0], K), k=draw(B, L, heads[1], K), v=draw(B, L, heads[2], V), dout=draw(B, L, H, V),
             rate=np.exp(rng.uniform(*np.log(rate), H)).astype(np.float32), dtype=dtype, S0=None, dlast=None, lens=None)
    if state:
        c["S0"], c["dlast"] = (rng.standard_normal((B, H, K, V)).astype(np.float32) for _ in range(2))
    if lens:
        c["lens"] = rng.integers(0, L + 1, B).astype(np.int32)
        c["lens"][0] = 0 if B > 1 else c["lens"][0]
        c["lens"][-1] = L
    return c


def upload(c):
    import torch
    t = {n: dev(c[n], c["dtype"]) for n in ("q", "k", "v", "dout")}
    t.update({n: dev(c[n]) for n in ("rate", "S0", "dlast")})
    t["lens"] = None if c["lens"] is None else torch.from_numpy(c["lens"]).cuda()
    return t


def limit(c, M, ref, rounded=True):
    L, H = c["q"].shape[1], len(c["rate"])
    C = (256 * float(min(c["rate"].max(), 1.0)) + 598 + 6 * (L / 32 + 1) + H) * U + (2.0 ** -16 if c["dtype"] == "bf16" else 0.0)
    return C * M + (2.0 ** -8 * np.abs(ref) if c["dtype"] == "bf16" and rounded else 0.0) + 1e-35


def close(got, ref, lim, what):
    g = host64(got)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    assert np.all(np.isfinite(g)), what
    bad = np.abs(g - ref) > lim
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[0], float(np.max(np.abs(g - ref) / lim)))


def check(mss, c, gradients=True, scale=0.3):
    t = upload(c)
    out, last = mss.linear_attention_fwd(t["q"], t["k"], t["v"], t["rate"], scale=scale, initial_state=t["S0"], seq_lens=t["lens"])
    s32 = float(np.float32(scale))
    args = (c["q"], c["k"], c["v"], c["rate"], s32)
    ref, rl = oracle.linear_attention(*args, c["S0"], c["lens"])
    M, Ml = oracle.linear_attention(*args, c["S0"], c["lens"], magnitude=True)
    close(out, ref, limit(c, M, ref), "out")
    close(last, rl, limit(c, Ml, rl, False), "last_state")
    if not gradients:
        return
    g = mss.linear_attention_bwd(t["q"], t["k"], t["v"], t["rate"], t["dout"], scale=scale, initial_state=t["S0"],
                                 seq_lens=t["lens"], dlast_state=t["dlast"], return_dinitial_state=True)
    args += (c["dout"], c["S0"], c["lens"], c["dlast"])
    ref, M = oracle.linear_attention_bwd(*args), oracle.linear_attention_bwd(*args, magnitude=True)
    for n in ("dq", "dk", "dv"):
        close(g[n], ref[n], limit(c, M[n], ref[n]), n)
    close(g["dinitial_state"], ref["dS0"], limit(c, M["dS0"], ref["dS0"], False), "dinitial_state")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 300])
def test_lengths(mss, L, dtype):
    check(mss, inputs(2, L, 3, 32, 48, dtype, state=L % 2 == 1, seed=L))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K,V", [(16, 16), (16, 128), (48, 64), (64, 64), (64, 80), (80, 112), (112, 16), (128, 64), (128, 128)])
def test_dims(mss, K, V, dtype):
    check(mss, inputs(1, 150, 2, K, V, dtype, state=True, seed=K + V))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads", [(1, 6, 6), (6, 1, 6), (6, 6, 1), (2, 3, 6), (1, 1, 1), (3, 3, 3), (6, 2, 2)])
def test_shared_heads(mss, heads, dtype):
    check(mss, inputs(2, 70, 6, 32, 64, dtype, heads=heads, lens=True, state=True, seed=sum(heads)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [40, 200, 700])
def test_sequences_of_different_lengths(mss, L, dtype):
    check(mss, inputs(5, L, 2, 64, 64, dtype, lens=True, state=True, seed=L + 1))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,H,K,V,lens", [(1, 2048, 1, 64, 64, False), (1, 1000, 2, 128, 128, False), (3, 1500, 1, 32, 80, True),
                                            (1, 5000, 1, 64, 32, False), (2, 777, 2, 16, 64, True)])
def test_few_heads_cut_in_segments(mss, B, L, H, K, V, lens, dtype):
    assert mss.linear_attention_scratch(B, L, H, H, H, H, K, V)[0] > 0  # there are segments
    check(mss, inputs(B, L, H, K, V, dtype, lens=lens, state=True, seed=L))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_head_in_many_segments(mss, dtype):
    """More segments than a wave has lanes, whose parts are joined by a kernel of their own."""
    check(mss, inputs(1, 12345, 1, 16, 32, dtype, state=True, seed=12))
    check(mss, inputs(2, 9000, 1, 32, 16, dtype, lens=True, state=True, seed=13))


@pytest.mark.parametrize("B,L,H,K,V,heads,dtype,gradients", [
    (11, 500, 40, 16, 16, (4, 4, 40), "bf16", True), (7, 500, 40, 16, 16, (4, 4, 40), "f32", True),
    (5, 1000, 110, 16, 128, None, "bf16", False)])
def test_batches_beyond_whole_rounds(mss, B, L, H, K, V, heads, dtype, gradients):
    """More blocks than find room at once: the last batches go in a launch of their own, cut finer."""
    check(mss, inputs(B, L, H, K, V, dtype, heads=heads, lens=True, state=True, seed=B + L), gradients=gradients)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decays_from_none_to_all(mss, dtype):
    c = inputs(2, 130, 7, 32, 32, dtype, state=True, lens=True, seed=4)
    c["rate"] = np.array([0.0, 1e-6, 0.5, 3.0, 90.0, 1e20, 3e38], dtype=np.float32)
    check(mss, c)
    # an infinite rate forgets everything: each step sees itself
    c["rate"][:] = np.inf
    t = upload(c)
    out, last = mss.linear_attention_fwd(t["q"], t["k"], t["v"], t["rate"], scale=1.0, initial_state=t["S0"])
    own = np.sum(c["q"].astype(np.float64) * c["k"], -1, keepdims=True) * c["v"]
    M = np.sum(np.abs(c["q"].astype(np.float64) * c["k"]), -1, keepdims=True) * np.abs(c["v"])
    close(out, own, limit(dict(c, rate=np.ones(7)), M, own), "out")
    kv = c["k"][:, -1, :, :, None].astype(np.float64) * c["v"][:, -1, :, None, :]
    close(last, kv, 64 * U * np.abs(kv) + 1e-35, "last")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_what_lies_past_the_ends_is_not_read(mss, dtype):
    import torch
    c = inputs(4, 200, 2, 32, 64, dtype, lens=True, state=True, seed=6)
    t = upload(c)
    run = lambda: (*mss.linear_attention_fwd(t["q"], t["k"], t["v"], t["rate"], initial_state=t["S0"], seq_lens=t["lens"]),  # noqa: E731
                   *mss.linear_attention_bwd(t["q"], t["k"], t["v"], t["rate"], t["dout"], initial_state=t["S0"], seq_lens=t["lens"],
                                             dlast_state=t["dlast"], return_dinitial_state=True).values())
    want = run()
    for b, n in enumerate(c["lens"]):
        for x in ("q", "k", "v", "dout"):
            t[x][b, n:] = float("nan")
    got = run()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert not want[0][0].any() and torch.equal(want[1][0], t["S0"][0])  # a sequence of no steps
    t["lens"] = torch.tensor([-5, 1000, 3, 200], dtype=torch.int32, device="cuda")  # clamped to 0 .. L
    t["dout"].nan_to_num_()
    [t[x].nan_to_num_() for x in ("q", "k", "v")]
    a = run()
    t["lens"] = torch.tensor([0, 200, 3, 200], dtype=torch.int32, device="cuda")
    assert all(torch.equal(x, y) for x, y in zip(a, run()))


def test_no_steps_and_no_batch(mss):
    import torch
    z = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    S0 = torch.randn(2, 3, 16, 32, device="cuda")
    out, last = mss.linear_attention_fwd(z(2, 0, 3, 16), z(2, 0, 3, 16), z(2, 0, 3, 32), z(3), initial_state=S0)
    assert out.shape == (2, 0, 3, 32) and torch.equal(last, S0)
    g = mss.linear_attention_bwd(z(2, 0, 3, 16), z(2, 0, 3, 16), z(2, 0, 3, 32), z(3), z(2, 0, 3, 32), dlast_state=S0,
                                 return_dinitial_state=True)
    assert torch.equal(g["dinitial_state"], S0) and g["dq"].numel() == 0
    assert not mss.linear_attention_fwd(z(2, 0, 3, 16), z(2, 0, 3, 16), z(2, 0, 3, 32), z(3))[1].any()
    assert mss.linear_attention_fwd(z(0, 5, 3, 16), z(0, 5, 3, 16), z(0, 5, 3, 32), z(3))[0].shape == (0, 5, 3, 32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,K,V,heads", [(1, 1, 16, 16, None), (3, 6, 48, 80, (2, 3, 6)), (2, 4, 128, 128, (4, 1, 2)),
                                           (64, 8, 128, 64, (1, 1, 8)), (2, 3, 112, 112, None)])
def test_one_token_chain_is_the_sequence(mss, B, H, K, V, heads, dtype):
    import torch
    L = 20
    c = inputs(B, L, H, K, V, dtype, heads=heads, state=True, seed=B + V)
    t = upload(c)
    state = t["S0"].clone()
    before = state._version
    outs = [mss.linear_attention_update(state, *(t[n][:, i].contiguous() for n in ("q", "k", "v")), t["rate"], scale=0.3)
            for i in range(L)]
    assert state._version > before
    args = (c["q"], c["k"], c["v"], c["rate"], float(np.float32(0.3)), c["S0"])
    ref, rl = oracle.linear_attention(*args)
    M, Ml = oracle.linear_attention(*args, magnitude=True)
    out = torch.stack(outs, 1)
    close(out, ref, (K + 8 * L + 8) * U * M + (2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0.0), "out")
    close(state, rl, 8 * (L + 1) * U * Ml, "state")
    bufs = [t[n][:, 0].contiguous() for n in ("q", "k", "v")]
    s2 = t["S0"].clone()
    bound = mss.LinearAttentionUpdateStep(s2, *bufs, t["rate"], scale=0.3)
    for i in range(L):
        [b.copy_(t[n][:, i]) for b, n in zip(bufs, ("q", "k", "v"))]
        assert torch.equal(bound(), outs[i])
    assert torch.equal(s2, state)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_token_of_many_states(mss, dtype):
    """States too large for the cache have the bits of the same states in parts."""
    import torch
    B, H, K, V = 37, 128, 64, 112
    tt = torch.bfloat16 if dtype == "bf16" else torch.float32
    state = torch.randn(B, H, K, V, device="cuda")
    assert state.numel() * 4 > 1 << 27
    q, k, v = (torch.randn(B, h, d, device="cuda").to(tt) for h, d in ((8, K), (H, K), (32, V)))
    rate = torch.rand(H, device="cuda")
    parts, outs = [], []
    for i in range(0, B, 5):
        s = state[i:i + 5].clone()
        outs.append(mss.linear_attention_update(s, q[i:i + 5], k[i:i + 5], v[i:i + 5], rate))
        parts.append(s)
    out = mss.linear_attention_update(state, q, k, v, rate)
    assert torch.equal(out, torch.cat(outs)) and torch.equal(state, torch.cat(parts))


def test_one_token_with_extreme_decays(mss):
    import torch
    S = torch.randn(1, 3, 16, 16, device="cuda")
    state, rate = S.clone(), torch.tensor([0.0, float("inf"), 1e-7], device="cuda")
    z = torch.zeros(1, 3, 16, device="cuda")
    mss.linear_attention_update(state, z, z, z, rate)
    assert torch.equal(state[0, 0], S[0, 0]) and not state[0, 1].any()
    assert torch.allclose(state[0, 2], S[0, 2] * (1 - 1e-7), rtol=1e-7, atol=0)


def test_same_bits_again_on_a_side_stream_and_in_a_graph(mss):
    import torch
    c = inputs(1, 1300, 4, 64, 64, "bf16", heads=(2, 4, 1), lens=True, state=True, seed=11)
    t = upload(c)

    def step():
        out, last = mss.linear_attention_fwd(t["q"], t["k"], t["v"], t["rate"], initial_state=t["S0"], seq_lens=t["lens"])
        g = mss.linear_attention_bwd(t["q"], t["k"], t["v"], t["rate"], t["dout"], initial_state=t["S0"], seq_lens=t["lens"],
                                     dlast_state=t["dlast"], return_dinitial_state=True)
        return [out, last, *g.values()]

    want = step()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(again, want))
    with torch.cuda.graph(graph, stream=side):
        got = step()
    for _ in range(3):
        [x.zero_() for x in got]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(step(), want))


def test_autograd(mss):
    import torch
    c = inputs(2, 90, 4, 32, 48, "f32", heads=(2, 1, 4), state=True, lens=True, seed=12)
    t = upload(c)
    leaves = {n: t[n].clone().requires_grad_() for n in ("q", "k", "v", "S0")}
    out, last = mss.LinearAttentionFunction.apply(leaves["q"], leaves["k"], leaves["v"], t["rate"], None, leaves["S0"], t["lens"])
    torch.autograd.backward([out, last], [t["dout"], t["dlast"]])
    g = mss.linear_attention_bwd(t["q"], t["k"], t["v"], t["rate"], t["dout"], initial_state=t["S0"], seq_lens=t["lens"],
                                 dlast_state=t["dlast"], return_dinitial_state=True)
    for n, m in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("S0", "dinitial_state")):
        assert torch.equal(leaves[n].grad, g[m]), n
    q = t["q"].clone().requires_grad_()  # the last state not used, no state before
    mss.LinearAttentionFunction.apply(q, t["k"], t["v"], t["rate"], 0.5)[0].backward(t["dout"])
    assert torch.equal(q.grad, mss.linear_attention_bwd(t["q"], t["k"], t["v"], t["rate"], t["dout"], scale=0.5)["dq"])
    with pytest.raises(ValueError, match="decay"):
        mss.LinearAttentionFunction.apply(t["q"], t["k"], t["v"], t["rate"].clone().requires_grad_())
    with pytest.raises(ValueError, match="gradient"):
        mss.linear_attention_update(last, *(t[n][:, 0].contiguous() for n in ("q", "k", "v")), t["rate"])


def test_offsets_past_31_bits(mss):
    """2^31 elements and more in each tensor, and short memories: the last steps' results depend on the steps near them."""
    import torch
    B, L, H, D = 1, 131136, 128, 128
    c = inputs(B, 96, H, D, D, "bf16", seed=13, rate=(2.0, 3.0))  # e^(-2 * 32) is far below a rounding
    q, k, v, d = (torch.zeros(B, L, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (d, "dout")):
        t[:, -96:] = dev(c[n], "bf16")
    rate = dev(c["rate"])
    out, last = mss.linear_attention_fwd(q, k, v, rate, scale=0.3)
    args = (c["q"], c["k"], c["v"], c["rate"], float(np.float32(0.3)))
    ref, rl = oracle.linear_attention(*args)
    M, Ml = oracle.linear_attention(*args, magnitude=True)
    close(out[:, -96:], ref, limit(dict(c, q=np.zeros((1, L))), M, ref), "out")
    close(last, rl, limit(dict(c, q=np.zeros((1, L))), Ml, rl, False), "last")
    assert not out[:, :-96].any()
    g = mss.linear_attention_bwd(q, k, v, rate, d, scale=0.3)
    args += (c["dout"],)
    ref, M = oracle.linear_attention_bwd(*args), oracle.linear_attention_bwd(*args, magnitude=True)
    for n in ("dq", "dk", "dv"):
        close(g[n][:, -96:], ref[n], limit(dict(c, q=np.zeros((1, L))), M[n], ref[n]), n)
        assert not g[n][:, :-96].any()
