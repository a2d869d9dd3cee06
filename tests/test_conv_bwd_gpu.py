"""GPU tests of the causal conv's gradients against the fp64 definition.

Tolerances, u = 2^-24, for |y| <= 8 (inputs and taps of order 1): y is off by K + 1 roundings of its
magnitude (at most 12), silu' changes by at most 0.5 per unit of y, the sigmoid in it by (|y| + 4) 2u and
that times (1 + |y|): at most (0.5 * 5 * 12 + 2 * 12 * 9) u = 246 u; with the products 256 u of the sums
with |dout| in dout's place and silu' at its greatest, 1.1.  dweight and dbias add up B L terms, at most
L / 64 + B + 16 additions in a row.  bf16 results add half a step, 2^-8 of the value."""
import numpy as np
import pytest

import oracle
from synth import round_to_bf16
from tests.gpu_helpers import dev, host64
from tests.test_gated_gpu import check, mss  # noqa: F401

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def inputs(B, D, L, K, dtype, seed):
    rng = np.random.default_rng(7000 + seed)
    rnd = round_to_bf16 if dtype == "bf16" else (lambda a: a)
    c = {n: rnd(rng.standard_normal(s).astype(np.float32)) for n, s in
         (("x", (B, D, L)), ("dout", (B, D, L)), ("st", (B, D, K - 1)), ("dfin", (B, D, K - 1)))}
    c["w"] = (0.5 * rng.standard_normal((D, K))).astype(np.float32)
    c["b"] = (0.5 * rng.standard_normal(D)).astype(np.float32)
    return dict(c, B=B, D=D, L=L, K=K, dtype=dtype)


def upload(c):
    return {n: dev(c[n], c["dtype"] if n in ("x", "dout", "st", "dfin") else "f32")
            for n in ("x", "dout", "st", "dfin", "w", "b")}


def check_all(c, g, silu, states, bias, what):
    st, dfin = (c["st"], c["dfin"]) if states else (None, None)
    ref = oracle.causal_conv1d_bwd(c["x"], c["w"], c["dout"], c["b"] if bias else None, st, silu, dfin)
    m = oracle.causal_conv1d_bwd(c["x"], c["w"], 1.1 * np.abs(c["dout"]), None, st, False,
                                 None if dfin is None else np.abs(dfin))
    r8 = 2.0 ** -8 if c["dtype"] == "bf16" else 0.0
    adds = (c["L"] / 64 + c["B"] + 16) * U
    check(g["dx"], ref["dx"], 256 * U * m["m_dx"] + r8 * np.abs(ref["dx"]) + 1e-37, what + " dx")
    check(g["dweight"], ref["dweight"], (256 * U + adds) * m["m_dweight"] + 1e-37, what + " dweight")
    check(g["dbias"], ref["dbias"], (256 * U + adds) * m["m_dbias"] + 1e-37, what + " dbias")
    if "dinitial_state" in g:
        check(g["dinitial_state"], ref["dstate"], 256 * U * m["m_dstate"] + r8 * np.abs(ref["dstate"]) + 1e-37,
              what + " dstate")


@pytest.mark.parametrize("B,D,L,K,dtype", [
    (2, 64, 256, 4, "f32"), (2, 64, 256, 4, "bf16"), (1, 7, 1, 4, "f32"), (2, 5, 2, 4, "bf16"), (1, 3, 3, 3, "f32"),
    (3, 5, 17, 4, "bf16"), (2, 48, 511, 3, "f32"), (2, 48, 512, 2, "bf16"), (1, 32, 513, 1, "f32"),
    (2, 6, 515, 4, "bf16"), (1, 3, 514, 4, "f32"), (4, 100, 1000, 4, "bf16"), (1, 2, 30001, 4, "f32"),
    (1, 1, 40960, 4, "bf16"), (5, 33, 1537, 2, "f32"),
    (300, 3, 50, 4, "f32"), (9000, 1, 30, 3, "bf16"), (6, 1030, 90, 4, "f32"), (2, 4100, 700, 4, "bf16"),
    (1, 8200, 40, 2, "f32"), (3, 2731, 520, 4, "bf16")])
@pytest.mark.parametrize("states,silu,bias", [(False, True, True), (True, True, False), (True, False, True)])
def test_conv_gradients(mss, B, D, L, K, dtype, states, silu, bias):  # noqa: F811
    import torch
    c = inputs(B, D, L, K, dtype, L + K)
    t = upload(c)
    kw = dict(bias=t["b"] if bias else None, initial_state=t["st"] if states else None, silu=silu,
              dfinal_state=t["dfin"] if states else None, return_dinitial_state=True)
    g = mss.causal_conv1d_bwd(t["x"], t["w"], t["dout"], **kw)
    check_all(c, g, silu, states, bias, f"conv bwd {B}x{D}x{L} K{K} {dtype} {states} {silu}")
    again = mss.causal_conv1d_bwd(t["x"], t["w"], t["dout"], **kw)
    assert all(torch.equal(g[n], again[n]) for n in g)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_that_start_anywhere(mss, dtype):  # noqa: F811
    import torch
    for L in (64, 520, 777):
        c = inputs(2, 6, L, 4, dtype, L)
        t = upload(c)
        for n in ("x", "dout"):
            flat = torch.empty(t[n].numel() + 1, dtype=t[n].dtype, device="cuda")
            flat[1:].copy_(t[n].reshape(-1))
            t[n] = flat[1:].view(t[n].shape)
        g = mss.causal_conv1d_bwd(t["x"], t["w"], t["dout"], bias=t["b"], initial_state=t["st"],
                                  dfinal_state=t["dfin"], return_dinitial_state=True)
        check_all(c, g, True, True, True, f"conv bwd off by one {L} {dtype}")


@pytest.mark.parametrize("B,D,L,dtype", [(4, 5120, 2048, "bf16"), (8, 1536, 2047, "f32")])
def test_layer_shapes(mss, B, D, L, dtype):  # noqa: F811
    c = inputs(B, D, L, 4, dtype, 1)
    t = upload(c)
    g = mss.causal_conv1d_bwd(t["x"], t["w"], t["dout"], bias=t["b"], initial_state=t["st"], dfinal_state=t["dfin"],
                              return_dinitial_state=True)
    ch = slice(None, None, 13)
    s = dict(c, **{n: c[n][:, ch] for n in ("x", "dout", "st", "dfin")}, w=c["w"][ch], b=c["b"][ch])
    check_all(s, {n: (v[ch] if n in ("dweight", "dbias") else v[:, ch]) for n, v in g.items()}, True, True, True,
              f"conv bwd layer {B}x{D}x{L} {dtype}")


def test_empty_sequences(mss):  # noqa: F811
    import torch
    c = inputs(2, 5, 0, 4, "f32", 1)
    t = upload(c)
    g = mss.causal_conv1d_bwd(t["x"], t["w"], t["dout"], bias=t["b"], initial_state=t["st"], dfinal_state=t["dfin"],
                              return_dinitial_state=True)
    assert torch.equal(g["dinitial_state"], t["dfin"]) and not g["dweight"].any() and not g["dbias"].any()
    n = torch.empty((0, 5, 9), device="cuda")
    g = mss.causal_conv1d_bwd(n, t["w"], n)
    assert not g["dweight"].any() and not g["dbias"].any()


def test_autograd_and_differences(mss):  # noqa: F811
    """The wrapper's gradients are the call's; and the loss moves along a direction as they say.  At
    e = 1/64 the quotient is off by its truncation, which the fp64 definition has at the same points, and by
    the outputs' rounding: y 5 u of its magnitude Y, silu (|y| + 8) u of itself, so
    (5 Y + (|y| + 8) |y|) u through |dout|, and the gradients by 256 u of their magnitudes."""
    import torch
    c = inputs(2, 6, 90, 4, "f32", 5)
    t = upload(c)
    leaves = [t[n].clone().requires_grad_() for n in ("x", "w", "b", "st")]
    out, fin = mss.CausalConv1dFunction.apply(*leaves)
    got = torch.autograd.grad((out * t["dout"]).sum() + (fin * t["dfin"]).sum(), leaves)
    g = mss.causal_conv1d_bwd(t["x"], t["w"], t["dout"], bias=t["b"], initial_state=t["st"], dfinal_state=t["dfin"],
                              return_dinitial_state=True)
    for u, n in zip(got, ("dx", "dweight", "dbias", "dinitial_state")):
        assert torch.equal(u, g[n]), n
    rng = np.random.default_rng(8)
    way = {n: rng.standard_normal(c[n].shape) for n in ("x", "w", "b", "st")}
    e, losses, exact, ps, noise = 1 / 64, [], [], [], 0.0
    for sgn in (1, -1):
        p = {n: (c[n] + sgn * e * way[n]).astype(np.float32) for n in way}
        o, f = mss.causal_conv1d_fwd(dev(p["x"]), dev(p["w"]), dev(p["b"]), initial_state=dev(p["st"]),
                                     return_final_state=True)
        losses.append(float((host64(o) * c["dout"]).sum() + (host64(f) * c["dfin"]).sum()))
        ro, rf = oracle.causal_conv1d(p["x"], p["w"], p["b"], state=p["st"])
        exact.append(float((ro * c["dout"]).sum() + (rf * c["dfin"]).sum()))
        y, _ = oracle.causal_conv1d(p["x"], p["w"], p["b"], state=p["st"], silu=False)
        Y, _ = oracle.causal_conv1d(*(np.abs(p[n]) for n in ("x", "w", "b")), state=np.abs(p["st"]), silu=False)
        noise += U * float((np.abs(c["dout"]) * (5 * Y + (np.abs(y) + 8) * np.abs(y))).sum())
        ps.append(p)
    pairs = (("dx", "x", "dx"), ("dweight", "w", "dweight"), ("dbias", "b", "dbias"), ("dinitial_state", "st", "dstate"))
    ref = oracle.causal_conv1d_bwd(c["x"], c["w"], c["dout"], c["b"], c["st"], True, c["dfin"])
    m = oracle.causal_conv1d_bwd(c["x"], c["w"], 1.1 * np.abs(c["dout"]), None, c["st"], False, np.abs(c["dfin"]))
    moved = {n: ps[0][n].astype(np.float64) - ps[1][n] for n in way}
    along = sum(float((host64(g[k]) * moved[n]).sum()) for k, n, _ in pairs)
    truncation = exact[0] - exact[1] - sum(float((ref[r] * moved[n]).sum()) for _, n, r in pairs)
    lim = noise + 256 * U * sum(float((m["m_" + r] * np.abs(moved[n])).sum()) for _, n, r in pairs)
    assert abs(losses[0] - losses[1] - along - truncation) <= lim, (losses, along, truncation, lim)
    assert abs(along) > 4 * (lim + abs(truncation))  # the direction says something


def test_chunks_give_the_whole_sequences_gradients(mss):  # noqa: F811
    """Two chunks trained with the window's gradient handed back equal one whole backward."""
    import torch
    c = inputs(2, 9, 1100, 4, "f32", 6)
    t = upload(c)
    whole = mss.causal_conv1d_bwd(t["x"], t["w"], t["dout"], bias=t["b"], initial_state=t["st"],
                                  return_dinitial_state=True)
    x1, x2 = t["x"][..., :501].contiguous(), t["x"][..., 501:].contiguous()
    d1, d2 = t["dout"][..., :501].contiguous(), t["dout"][..., 501:].contiguous()
    st = x1[..., -3:].contiguous()
    g2 = mss.causal_conv1d_bwd(x2, t["w"], d2, bias=t["b"], initial_state=st, return_dinitial_state=True)
    g1 = mss.causal_conv1d_bwd(x1, t["w"], d1, bias=t["b"], initial_state=t["st"],
                               dfinal_state=g2["dinitial_state"], return_dinitial_state=True)
    c["dfin"] = np.zeros_like(c["dfin"])
    check_all(c, dict(dx=torch.cat([g1["dx"], g2["dx"]], -1), dweight=g1["dweight"] + g2["dweight"],
                      dbias=g1["dbias"] + g2["dbias"], dinitial_state=g1["dinitial_state"]), True, True, True,
              "conv bwd in chunks")
    assert torch.equal(whole["dinitial_state"], g1["dinitial_state"])


def test_more_than_2_to_the_31_elements(mss):  # noqa: F811
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    B, D, L = 3, 350, 2100000
    x, d = (torch.empty((B, D, L), dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    w = torch.randn((D, 4), generator=g, device="cuda")
    got = mss.causal_conv1d_bwd(x, w, d)
    part = mss.causal_conv1d_bwd(x[-1:, -2:].contiguous(), w[-2:].contiguous(), d[-1:, -2:].contiguous())
    assert torch.equal(got["dx"][-1:, -2:], part["dx"])


def test_captured_without_a_call_before_and_replayed(mss):  # noqa: F811
    import torch
    t = upload(inputs(2, 24, 1500, 4, "bf16", 11))
    torch.cuda.synchronize()

    def body():
        g = mss.causal_conv1d_bwd(t["x"], t["w"], t["dout"], bias=t["b"], initial_state=t["st"],
                                  dfinal_state=t["dfin"], return_dinitial_state=True)
        return list(g.values())

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        res = body()
    for rep in range(3):
        n = upload(inputs(2, 24, 1500, 4, "bf16", 12 + rep))
        for k in t:
            t[k].copy_(n[k])
        want = [v.clone() for v in body()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(res, want)), rep
