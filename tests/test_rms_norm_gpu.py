"""GPU tests of the RMS norm (output in the activations' type and in e4m3, gradients) against the fp64 definition.

Tolerances, with u = 2^-24 (half a step of fp32), for rows of up to 16384 columns:
  - the sum of squares: a lane adds up to 16 squares in a row, then 6 steps over the wave and 6 over the waves: 28 u,
    all terms positive; its root halves that; mean, eps, root and reciprocal 4 u: rstd 18 u.
  - out = z r w: two more roundings: 20 u.  In bf16 half a step more, 2^-8 of the value.
  - in e4m3 the scale is the greatest such value / 448 (22 u), the quotient 24 u off, its rounding half a step: 2^-4 of
    the value, or 2^-10 scales below the type's normal numbers.
  - dz: z r 19 u, times w dout 2 u, its mean 28 u more, r 18 u: 70 u of the magnitudes.
  - dweight adds its terms (21 u each) over rows: R u at most, and 70 in the joins."""
import numpy as np
import pytest

import oracle
from synth import round_to_bf16
from tests.gpu_helpers import dev, host64

pytestmark = pytest.mark.gpu
U, HALF = 2.0 ** -24, {"f32": 0.0, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def mss():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_06_amd as m
    m.load_library()
    return m


def inputs(shape, dtype, residual, seed=0, scale=1.0):
    rng = np.random.default_rng(7000 + seed)

    def draw(t, s=1.0):
        a = (rng.standard_normal(shape) * s).astype(np.float32)
        return round_to_bf16(a) if t == "bf16" else a

    c = dict(x=draw(dtype, scale), w=rng.uniform(0.5, 1.5, shape[-1]).astype(np.float32), dout=draw(dtype), stream=None,
             dstream=None, dtype=dtype, residual=residual)
    if residual:
        c["stream"], c["dstream"] = draw(residual, 4.0), draw(residual)
    return c


def stream_of(c):
    """The stream after the addition, as it is written: fp32 arithmetic, then the stream's type."""
    if c["stream"] is None:
        return c["x"]
    z = c["x"] + c["stream"]
    return round_to_bf16(z) if c["residual"] == "bf16" else z


def close(got, ref, lim, what):
    g = host64(got).reshape(ref.shape)
    assert np.all(np.isfinite(g)), what
    bad = np.abs(g - ref) > lim
    assert not bad.any(), (what, int(bad.sum()), float(np.max(np.abs(g - ref) / (lim + 1e-300))))


WIDTHS = [1, 3, 8, 64, 127, 768, 2049, 2560, 5120, 8192, 8193, 16384, 16383]
TYPES = [("f32", None), ("f32", "f32"), ("bf16", None), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "bf16")]


def flat(a):
    return a.reshape(-1, a.shape[-1])


@pytest.mark.parametrize("dtype,residual", TYPES)
@pytest.mark.parametrize("W", WIDTHS)
def test_forward_and_gradients(mss, W, dtype, residual):
    R = 5 if W > 1000 else 37
    c = inputs((R, W), dtype, residual, W)
    z = stream_of(c)
    out, stream, rstd = mss.rms_norm_fwd_save(dev(c["x"], dtype), dev(c["w"]), residual=dev(c["stream"], residual), eps=1e-5)
    ref, r = oracle.rms_norm(z, c["w"], float(np.float32(1e-5)))
    close(out, ref, (20 * U + HALF[dtype]) * np.abs(ref) + 1e-37, "out")
    close(rstd, r, 18 * U * r, "rstd")
    if residual:
        assert np.array_equal(host64(stream), z.astype(np.float64))
    else:
        assert stream is None
    out2, _ = mss.rms_norm_fwd(dev(c["x"], dtype), dev(c["w"]), residual=dev(c["stream"], residual), eps=1e-5)
    assert np.array_equal(host64(out), host64(out2))
    g = mss.rms_norm_bwd(dev(z, residual or dtype), dev(c["w"]), rstd, dev(c["dout"], dtype),
                         dresidual_out=dev(c["dstream"], residual))
    ref = oracle.rms_norm_bwd(z, c["w"], float(np.float32(1e-5)), c["dout"], c["dstream"])
    lim = 70 * U * ref["m_dz"] + 1e-37
    close(g["dx"], ref["dz"], lim + HALF[dtype] * np.abs(ref["dz"]), "dx")
    close(g["dweight"], ref["dweight"], (R + 91) * U * ref["m_dweight"] + 1e-37, "dweight")
    if residual:
        close(g["dresidual"], ref["dz"], lim + HALF[residual] * np.abs(ref["dz"]), "dresidual")
        assert (g["dresidual"] is g["dx"]) == (residual == dtype)
    else:
        assert "dresidual" not in g


@pytest.mark.parametrize("R,W", [(1, 2560), (4096, 64), (5000, 1000), (20000, 40), (1000, 4100)])
def test_many_rows_and_their_weights(mss, R, W):
    c = inputs((R, W), "bf16", "f32", R)
    z = stream_of(c)
    out, stream, rstd = mss.rms_norm_fwd_save(dev(c["x"], "bf16"), dev(c["w"]), residual=dev(c["stream"]))
    g = [mss.rms_norm_bwd(stream, dev(c["w"]), rstd, dev(c["dout"], "bf16"), dresidual_out=dev(c["dstream"]))
         for _ in range(2)]
    ref, _ = oracle.rms_norm(z, c["w"], 1e-5)
    close(out, ref, (21 * U + 2.0 ** -8) * np.abs(ref) + 1e-37, "out")
    ref = oracle.rms_norm_bwd(z, c["w"], 1e-5, c["dout"], c["dstream"])
    close(g[0]["dresidual"], ref["dz"], 71 * U * ref["m_dz"], "dresidual")
    close(g[0]["dweight"], ref["dweight"], (R + 92) * U * ref["m_dweight"], "dweight")
    for n in g[0]:
        assert np.array_equal(host64(g[0][n]), host64(g[1][n])), n  # the same bits again


@pytest.mark.parametrize("group", [None, 128])
@pytest.mark.parametrize("dtype,residual", [("f32", None), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("W", [1, 64, 127, 128, 129, 1000, 2560, 8200, 16384])
def test_eight_bits(mss, W, dtype, residual, group):
    import torch
    c = inputs((2, 3, W), dtype, residual, W + 1)
    c["w"][W // 2] = 0.0
    q, scales, stream = mss.rms_norm_fwd_e4m3(dev(c["x"], dtype), dev(c["w"]), residual=dev(c["stream"], residual), group=group)
    assert q.dtype == torch.float8_e4m3fn and q.shape == c["x"].shape
    assert scales.shape == (2, 3, 1 if group is None else -(-W // 128))
    ref, _ = oracle.rms_norm(flat(stream_of(c)), c["w"], float(np.float32(1e-5)))
    n = group or W
    most = np.stack([np.abs(ref[:, i:i + n]).max(-1) for i in range(0, W, n)], -1)
    want = np.maximum(most, 2.0 ** -100) / 448
    s = host64(scales).reshape(want.shape)
    assert np.all(np.abs(s - want) <= 22 * U * want)
    wide = np.repeat(s, n, -1)[:, :W]
    got = q.float().double().cpu().numpy().reshape(ref.shape) * wide
    lim = np.maximum((2.0 ** -4 + 24 * U) * np.abs(ref), 2.0 ** -10 * wide * (1 + 2.0 ** -10))
    assert np.all(np.isfinite(got)) and np.all(np.abs(got - ref) <= lim)
    assert np.max(np.abs(q.float().cpu().numpy())) == 448.0 or not ref.any()  # the type's range is used
    # nearest even, away from ties: what torch's rounding of the same quotient gives
    quo = ref / wide
    near = torch.from_numpy(quo).float().to(torch.float8_e4m3fn).float().numpy()
    far = torch.from_numpy(quo * (1 + 64 * U)).float().to(torch.float8_e4m3fn).float().numpy()
    low = torch.from_numpy(quo * (1 - 64 * U)).float().to(torch.float8_e4m3fn).float().numpy()
    sure = (near == far) & (near == low)
    assert np.array_equal(q.float().cpu().numpy().reshape(ref.shape)[sure], near[sure])


def test_zero_rows_infinities_and_nan(mss):
    import torch
    x = torch.ones(4, 300, device="cuda")
    x[0] = 0.0
    x[1, 7] = float("nan")
    x[2, 5] = float("inf")
    w = torch.ones(300, device="cuda")
    out, _, rstd = mss.rms_norm_fwd_save(x, w)
    assert not out[0].any() and torch.isnan(out[1]).all() and torch.isnan(rstd[1])
    assert torch.isnan(out[2, 5]) and not torch.nan_to_num(out[2]).any()
    assert abs(float(out[3, 0]) - 1.0) < 1e-5 and torch.isfinite(out[3]).all()
    q, s, _ = mss.rms_norm_fwd_e4m3(x, w)
    assert not q[0].float().any() and float(s[0, 0]) == np.float32(2.0 ** -100) / np.float32(448)
    assert torch.isnan(q[1].float()).all() and torch.isnan(q[2, 5].float()) and (q[3].float() == 448).all()


def test_in_place_stream_unaligned_views_and_no_rows(mss):
    import torch
    c = inputs((6, 515), "bf16", "f32", 3)
    want, ws, _ = mss.rms_norm_fwd_save(dev(c["x"], "bf16"), dev(c["w"]), residual=dev(c["stream"]))
    stream = dev(c["stream"])
    out, same = mss.rms_norm_fwd(dev(c["x"], "bf16"), dev(c["w"]), residual=stream, residual_out=stream)
    assert same is stream and torch.equal(stream, ws) and torch.equal(out, want)
    big = torch.zeros(6 * 515 + 9, dtype=torch.bfloat16, device="cuda")
    view = big[3:3 + 6 * 515].view(6, 515)
    view.copy_(dev(c["x"], "bf16"))
    off = torch.empty(6 * 515 + 9, dtype=torch.float8_e4m3fn, device="cuda")[5:5 + 6 * 515].view(6, 515)
    out, _ = mss.rms_norm_fwd(view, dev(c["w"]), residual=dev(c["stream"]))
    assert torch.equal(out, want)
    q, s, _ = mss.rms_norm_fwd_e4m3(view, dev(c["w"]), residual=dev(c["stream"]), out=off)
    q2, s2, _ = mss.rms_norm_fwd_e4m3(dev(c["x"], "bf16"), dev(c["w"]), residual=dev(c["stream"]))
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2) and not big[-6:].any()
    none = torch.empty(0, 515, device="cuda")
    assert mss.rms_norm_fwd(none, dev(c["w"]))[0].shape == (0, 515)
    g = mss.rms_norm_bwd(none, dev(c["w"]), torch.empty(0, device="cuda"), none)
    assert g["dweight"].shape == (515,) and not g["dweight"].any()


def test_rows_past_31_bits_of_elements(mss):
    import torch
    R, W = 131080, 16384
    x = torch.zeros(R, W, dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, 131071, 131072, R - 1]
    c = inputs((len(rows), W), "bf16", None, 9)
    x[rows] = dev(c["x"], "bf16")
    out, _, rstd = mss.rms_norm_fwd_save(x, dev(c["w"]))
    ref, r = oracle.rms_norm(c["x"], c["w"], 1e-5)
    close(out[rows], ref, (21 * U + 2.0 ** -8) * np.abs(ref) + 1e-37, "out")
    assert not out[2:131071].any()
    dout = torch.zeros_like(x)
    dout[rows] = dev(c["dout"], "bf16")
    g = mss.rms_norm_bwd(x, dev(c["w"]), rstd, dout)
    ref = oracle.rms_norm_bwd(c["x"], c["w"], 1e-5, c["dout"])
    close(g["dx"][rows], ref["dz"], 71 * U * ref["m_dz"] + 2.0 ** -8 * np.abs(ref["dz"]), "dx")
    close(g["dweight"], ref["dweight"], (R + 92) * U * ref["m_dweight"] + 1e-37, "dweight")


def test_graph_stream_bound_step_and_autograd(mss):
    import torch
    c = inputs((8, 1536), "bf16", "f32", 5)
    x, w, s0 = dev(c["x"], "bf16"), dev(c["w"]), dev(c["stream"])
    dout, ds = dev(c["dout"], "bf16"), dev(c["dstream"])

    def step(stream):
        out, z, rstd = mss.rms_norm_fwd_save(x, w, residual=stream)
        return (out, z, *mss.rms_norm_bwd(z, w, rstd, dout, dresidual_out=ds).values(),
                *mss.rms_norm_fwd_e4m3(x, w, residual=stream, group=128)[:2])

    want = step(s0)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        got = step(s0)
    for _ in range(3):
        for t in got:
            t.view(torch.uint8).zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
        step(s0)
    stream = s0.clone()
    bound = mss.RMSNormStep(x, w, residual=stream)
    before = stream._version
    for _ in range(3):
        prior = stream.clone()
        out = bound()
        a, b = mss.rms_norm_fwd(x, w, residual=prior)
        assert torch.equal(out, a) and torch.equal(stream, b)
    assert stream._version > before
    leaves = [t.clone().requires_grad_() for t in (x, w, s0)]
    out, z = mss.RMSNormFunction.apply(*leaves)
    torch.autograd.backward([out, z], [dout, ds])
    assert torch.equal(leaves[0].grad, want[2]) and torch.equal(leaves[1].grad, want[3])
    assert torch.equal(leaves[2].grad, want[4])
    x2 = x.clone().requires_grad_()
    out, none = mss.RMSNormFunction.apply(x2, w)
    assert none is None
    out.backward(dout)
    r = mss.rms_norm_fwd_save(x, w)[2]
    assert torch.equal(x2.grad, mss.rms_norm_bwd(x, w, r, dout)["dx"])


def test_more_rows_than_blocks(mss):
    import torch
    R, W = (1 << 21) + 5, 9
    x, s = torch.randn(R, W, device="cuda"), torch.randn(R, W, device="cuda")
    w = torch.randn(W, device="cuda")
    out, z = mss.rms_norm_fwd(x, w, residual=s)
    z64 = z.double()
    assert torch.equal(z, x + s)
    want = z64 * torch.rsqrt(z64.square().mean(-1, keepdim=True) + float(np.float32(1e-5))) * w.double()
    assert bool(((out - want).abs() <= 20 * U * want.abs()).all())
    q, scales, _ = mss.rms_norm_fwd_e4m3(x, w, residual=s)
    assert bool(((q.double() * scales - want).abs() <= (2.0 ** -4 + 30 * U) * want.abs() + 2.0 ** -10 * scales).all())
