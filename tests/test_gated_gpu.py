"""GPU tests of the gated scan, its gradients and its one-token step against the fp64 definitions.

Tolerances, with u = 2^-24 (half a step of fp32) and every term taken with its magnitude (the scan of
|x| and |h0|; all its weights are positive, so M = oracle(|x|, |h0|) bounds every partial sum):
  - a gate: e^-f carries the rounding of f log2 e, |f| u, and a few u of exp2, 1 + e and the
    reciprocal: (|f| + 8) u, and |f| <= 6 for these inputs, so 14 u; s = rate r two more; a = e^-s adds
    s (16 u) + 2 u; m = sqrt(q) half of q's error (16 u from s, 8 u from the series) + 2 u: 14 u; the
    input term m p x then 14 + 14 + 4 = 32 u.
  - the state: over the steps it remembers, sum of s is about 1, so the a of all of them add
    16 u; their own rounding and the multiply-add add at most 3 u a step, over at most n = L steps (and the
    lane and tile joins a few more): C = (56 + 3 n) u of M.
  - a gradient is a product of the adjoint (C of its magnitude), the state before (C of its), and local
    factors (64 u): (2 C + 64 u) of the magnitude sums of the gradients formula.
  - drate adds up B L terms in fp32, at most B + L / 64 + 16 additions in a row: that many u more.
A bf16 result adds half a bf16 step, 2^-8 of its value."""
import numpy as np
import pytest

import oracle
from tests.gpu_helpers import dev, host64
from synth import round_to_bf16

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


def inputs(B, D, L, dtype, seed, lens=False, h0=False, lo=0.9, hi=0.999):
    rng = np.random.default_rng(5000 + seed)
    rnd = round_to_bf16 if dtype == "bf16" else (lambda a: a)
    c = dict(B=B, D=D, L=L, dtype=dtype)
    for n in ("x", "f", "i", "dout"):
        c[n] = rnd(np.clip(rng.standard_normal((B, D, L)), -6, 6).astype(np.float32))
    c["rate"] = (-np.log(rng.uniform(lo, hi, D))).astype(np.float32)
    c["h0"] = rng.standard_normal((B, D)).astype(np.float32) if h0 else None
    c["dlast"] = rng.standard_normal((B, D)).astype(np.float32) if h0 else None
    c["lens"] = None
    if lens:
        c["lens"] = rng.integers(0, L + 1, B).astype(np.int32)
        c["lens"][0] = 0 if B > 1 else c["lens"][0]
        c["lens"][-1] = L
    return c


def upload(c):
    import torch
    t = {n: dev(c[n], c["dtype"]) for n in ("x", "f", "i", "dout")}
    t.update({n: dev(c[n]) for n in ("rate", "h0", "dlast")})
    t["lens"] = None if c["lens"] is None else torch.from_numpy(c["lens"]).cuda()
    return t


def check(got, ref, lim, what):
    g = host64(got)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    assert np.all(np.isfinite(g)), what
    err = np.abs(g - ref)
    if err.size:
        ratio = float((err / lim).max())
        assert ratio <= 1.0, (what, ratio, float(err.max()))


def limits(c, M, ref, rounded=True):
    C = (56 + 3 * c["L"]) * U
    return C * M + (2.0 ** -8 * np.abs(ref) if c["dtype"] == "bf16" and rounded else 0.0) + 1e-37


def check_forward(c, out, last, saved, what):
    ref, rl, before = oracle.gated_scan(c["x"], c["f"], c["i"], c["rate"], c["h0"], c["lens"])
    ab = None if c["h0"] is None else np.abs(c["h0"])
    M, Ml, Mb = oracle.gated_scan(np.abs(c["x"]), c["f"], c["i"], c["rate"], ab, c["lens"])
    check(out, ref, limits(c, M, ref), what + " out")
    check(last, rl, limits(c, Ml, rl, False), what + " last")
    if saved is not None and c["L"]:
        check(saved, before[..., ::512], limits(c, Mb[..., ::512], before[..., ::512], False), what + " saved")


def check_grads(c, g, what):
    ref = oracle.gated_scan_bwd(c["x"], c["f"], c["i"], c["rate"], c["dout"], c["h0"], c["lens"], c["dlast"])
    ab = {n: None if c[n] is None else np.abs(c[n]) for n in ("x", "dout", "h0", "dlast")}
    mag = oracle.gated_scan_bwd(ab["x"], c["f"], c["i"], c["rate"], ab["dout"], ab["h0"], c["lens"], ab["dlast"])
    C = (2 * (56 + 3 * c["L"]) + 64) * U
    for n, r in (("dx", "dx"), ("dfgate", "dfgate"), ("digate", "digate"), ("dinitial_state", "dh0")):
        if n in g:
            bf = c["dtype"] == "bf16" and n != "dinitial_state"
            check(g[n], ref[r], C * mag["m_" + r] + (2.0 ** -8 * np.abs(ref[r]) if bf else 0) + 1e-37, f"{what} {n}")
    adds = c["B"] + c["L"] / 64 + 16
    check(g["drate"], ref["drate"], (C + adds * U) * mag["m_drate"] + 1e-37, what + " drate")


SHAPES = [(2, 64, 256, "f32"), (2, 64, 256, "bf16"), (1, 3, 1, "f32"), (1, 5, 1, "bf16"), (3, 5, 7, "f32"),
          (2, 70, 511, "bf16"), (2, 70, 512, "bf16"), (2, 7, 513, "f32"), (1, 1, 2047, "f32"), (2, 33, 1500, "bf16"),
          (1, 9, 5000, "f32"), (2, 11, 4104, "bf16"), (1, 2, 20001, "f32"), (1, 1, 40960, "bf16"),
          (1, 130, 9000, "f32"), (1, 3, 70001, "f32"), (2, 20, 66048, "bf16"), 
          (3, 1030, 4097, "f32"), (2, 2100, 1100, "f32"), (1, 5000, 600, "bf16"),
          (300, 3, 50, "f32"), (2100, 2, 40, "bf16"), (700, 3, 1100, "f32"), (6, 1030, 90, "f32")]


@pytest.mark.parametrize("B,D,L,dtype", SHAPES)
@pytest.mark.parametrize("lens,h0", [(False, False), (True, True)])
def test_forward_and_gradients(mss, B, D, L, dtype, lens, h0):
    import torch
    c = inputs(B, D, L, dtype, B + D + L, lens, h0)
    t = upload(c)
    what = f"gated {B}x{D}x{L} {dtype} lens={lens} h0={h0}"
    out, last = mss.gated_scan_fwd(t["x"], t["f"], t["i"], t["rate"], initial_state=t["h0"], seq_lens=t["lens"])
    out2, last2, saved = mss.gated_scan_fwd_save(t["x"], t["f"], t["i"], t["rate"], initial_state=t["h0"],
                                                 seq_lens=t["lens"])
    assert torch.equal(out, out2) and torch.equal(last, last2)
    check_forward(c, out, last, saved, what)
    kw = dict(seq_lens=t["lens"], dlast_state=t["dlast"], return_dinitial_state=True)
    g = mss.gated_scan_bwd(t["x"], t["f"], t["i"], t["rate"], t["dout"], saved_states=saved, **kw)
    check_grads(c, g, what)
    # the states run again instead of kept, and the whole call again: the same bits
    for again in (mss.gated_scan_bwd(t["x"], t["f"], t["i"], t["rate"], t["dout"], initial_state=t["h0"], **kw),
                  mss.gated_scan_bwd(t["x"], t["f"], t["i"], t["rate"], t["dout"], saved_states=saved, **kw)):
        for n in g:
            assert torch.equal(g[n], again[n]), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_that_start_anywhere(mss, dtype):
    """Tensors one element past a 16-byte boundary, of row lengths that are whole vectors and not."""
    import torch
    for L in (64, 520, 777, 2040):
        c = inputs(2, 6, L, dtype, L, True, True)
        t = upload(c)
        for n in ("x", "f", "i", "dout"):
            flat = torch.empty(t[n].numel() + 1, dtype=t[n].dtype, device="cuda")
            flat[1:].copy_(t[n].reshape(-1))
            t[n] = flat[1:].view(t[n].shape)
        out, last, saved = mss.gated_scan_fwd_save(t["x"], t["f"], t["i"], t["rate"], initial_state=t["h0"],
                                                   seq_lens=t["lens"])
        check_forward(c, out, last, saved, f"gated off by one {L} {dtype}")
        g = mss.gated_scan_bwd(t["x"], t["f"], t["i"], t["rate"], t["dout"], seq_lens=t["lens"], saved_states=saved,
                               dlast_state=t["dlast"], return_dinitial_state=True)
        check_grads(c, g, f"gated off by one {L} {dtype}")


@pytest.mark.parametrize("dtype,L", [("f32", 1300), ("bf16", 1304)])
def test_nothing_past_a_sequences_end_matters(mss, dtype, L):
    """NaN and infinities in every input past the lengths: outputs and gradients are those of zeros
    there, bit for bit; lengths out of range are clamped."""
    import torch
    c = inputs(4, 5, L, dtype, 3, True, True)
    c["lens"] = np.array([0, 1, 700, L], np.int32)
    t = upload(c)
    runs = []
    for fill in (0.0, float("nan"), float("inf")):
        for n in ("x", "f", "i", "dout"):
            for b, k in enumerate(c["lens"]):
                t[n][b, :, k:] = fill
        lens = torch.tensor([-5, 1, 700, 2 ** 30], dtype=torch.int32, device="cuda") if fill else t["lens"]
        out, last, saved = mss.gated_scan_fwd_save(t["x"], t["f"], t["i"], t["rate"], initial_state=t["h0"],
                                                   seq_lens=lens)
        g = mss.gated_scan_bwd(t["x"], t["f"], t["i"], t["rate"], t["dout"], seq_lens=lens, saved_states=saved,
                               dlast_state=t["dlast"], return_dinitial_state=True)
        runs.append((out, last, saved, *g.values()))
        assert all(torch.isfinite(v.float()).all() for v in runs[-1])
        assert torch.equal(last[0], t["h0"][0]) and torch.equal(g["dinitial_state"][0], t["dlast"][0])
        for b, k in enumerate(c["lens"]):
            assert not any(v[b, :, k:].any() for v in (out, g["dx"], g["dfgate"], g["digate"]))
    for other in runs[1:]:
        assert all(torch.equal(u, v) for u, v in zip(runs[0], other))


def test_gates_at_their_ends(mss):
    """Gates far open and far closed, infinite ones, and decays from 1e-7 to 60 a step."""
    import torch
    c = inputs(1, 8, 600, "f32", 9, False, True)
    c["rate"] = np.array([1e-7, 1e-4, 0.01, 0.124, 0.126, 1.0, 10.0, 60.0], np.float32)
    rng = np.random.default_rng(1)
    c["f"] = rng.choice(np.array([-200, -60, -10, 0, 10, 60, 200, -np.inf, np.inf], np.float32), c["f"].shape)
    c["i"] = rng.choice(np.array([-200, -60, -10, 0, 10, 60, 200, -np.inf, np.inf], np.float32), c["i"].shape)
    t = upload(c)
    out, last, saved = mss.gated_scan_fwd_save(t["x"], t["f"], t["i"], t["rate"], initial_state=t["h0"])
    # |f| up to 10 between the flat ends; where e^-f underflows or overflows (|f| >= 60) r is 0 or 1 to
    # within e^-60 = 9e-27, sqrt of rate times which is below 1e-12 a step and 1e-9 in all
    with np.errstate(over="ignore"):
        ref, rl, _ = oracle.gated_scan(c["x"], c["f"], c["i"], c["rate"], c["h0"])
        M, Ml, _ = oracle.gated_scan(np.abs(c["x"]), c["f"], c["i"], c["rate"], np.abs(c["h0"]))
        check(out, ref, limits(c, M, ref) + 1e-9, "gates at their ends out")
        check(last, rl, limits(c, Ml, rl) + 1e-9, "gates at their ends last")
        g = mss.gated_scan_bwd(t["x"], t["f"], t["i"], t["rate"], t["dout"], saved_states=saved)
        r = oracle.gated_scan_bwd(c["x"], c["f"], c["i"], c["rate"], c["dout"], c["h0"])
        m = oracle.gated_scan_bwd(np.abs(c["x"]), c["f"], c["i"], c["rate"], np.abs(c["dout"]), np.abs(c["h0"]))
    C = (2 * (56 + 3 * 600) + 64) * U
    for n in ("dx", "dfgate", "digate"):
        check(g[n], r[n], C * m["m_" + n] + 1e-9, "gates at their ends " + n)
    # through sqrt(1 - a^2) the gradient to rate grows like r / sqrt(2 rate r): terms whose r is below
    # fp32's range are left out, sqrt(1e-38 / (2 rate)) < 1e-15 each
    check(g["drate"], r["drate"], (C + 64 * U) * m["m_drate"] + 1e-9, "gates at their ends drate")
    z = mss.gated_scan_bwd(t["x"], t["f"], t["i"], torch.zeros_like(t["rate"]), t["dout"], initial_state=t["h0"])
    assert all(torch.isfinite(v).all() for v in z.values()) and not z["dx"].any()


def test_empty_sequences_and_channels(mss):
    import torch
    e = torch.empty((3, 4, 0), device="cuda")
    h0, rate = torch.randn((3, 4), device="cuda"), torch.ones(4, device="cuda")
    out, last, saved = mss.gated_scan_fwd_save(e, e, e, rate, initial_state=h0)
    assert out.shape == (3, 4, 0) and saved.shape == (3, 4, 0) and torch.equal(last, h0)
    g = mss.gated_scan_bwd(e, e, e, rate, e, dlast_state=h0, return_dinitial_state=True, saved_states=saved)
    assert torch.equal(g["dinitial_state"], h0) and not g["drate"].any()
    n = torch.empty((0, 4, 9), device="cuda")
    out, last = mss.gated_scan_fwd(n, n, n, rate)
    assert out.shape == (0, 4, 9) and last.shape == (0, 4)
    assert not mss.gated_scan_bwd(n, n, n, rate, n)["drate"].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_chunks_and_single_tokens_continue_a_sequence(mss, dtype):
    """A sequence in chunks, each from the last one's state, and token by token: both within the
    forward's limits of the whole."""
    import torch
    c = inputs(2, 40, 600, dtype, 21, False, True)
    t = upload(c)
    st, parts = t["h0"], []
    for lo, hi in ((0, 1), (1, 257), (257, 600)):
        o, st = mss.gated_scan_fwd(*(t[n][..., lo:hi].contiguous() for n in ("x", "f", "i")), t["rate"],
                                   initial_state=st)
        parts.append(o)
    check_forward(c, torch.cat(parts, -1), st, None, f"gated in chunks {dtype}")
    st, parts = t["h0"].clone(), []
    step = None
    bufs = [t[n][..., 0].contiguous() for n in ("x", "f", "i")]
    for k in range(600):
        for b, n in zip(bufs, ("x", "f", "i")):
            b.copy_(t[n][..., k])
        if k % 2:
            parts.append(mss.gated_state_update(st, *bufs, t["rate"]))
        else:
            step = step or mss.GatedUpdateStep(st, *bufs, t["rate"])
            parts.append(step().clone())
    check_forward(c, torch.stack(parts, -1), st, None, f"gated by tokens {dtype}")


@pytest.mark.parametrize("B,D,dtype", [(1, 1, "f32"), (1, 1536, "f32"), (64, 5120, "bf16"), (3, 333, "bf16"),
                                       (2, 4097, "f32")])
def test_single_token(mss, B, D, dtype):
    c = inputs(B, D, 1, dtype, D, False, True)
    t = upload(c)
    st = t["h0"].clone()
    out = mss.gated_state_update(st, t["x"][..., 0].contiguous(), t["f"][..., 0].contiguous(),
                                 t["i"][..., 0].contiguous(), t["rate"])
    ref = oracle.gated_state_update(c["h0"], c["x"][..., 0], c["f"][..., 0], c["i"][..., 0], c["rate"])
    M = oracle.gated_state_update(np.abs(c["h0"]), np.abs(c["x"][..., 0]), c["f"][..., 0], c["i"][..., 0], c["rate"])
    check(st, ref, limits(c, M, ref, False), f"gated token {B}x{D} {dtype} state")
    check(out, ref, limits(c, M, ref), f"gated token {B}x{D} {dtype} out")


def test_autograd_gives_the_calls_gradients(mss):
    import torch
    c = inputs(2, 12, 700, "f32", 31, True, True)
    t = upload(c)
    leaves = [t[n].clone().requires_grad_() for n in ("x", "f", "i", "rate", "h0")]
    out, last = mss.GatedScanFunction.apply(*leaves, t["lens"])
    # dout arrives as an expanded tensor, dlast with strides: both are laid out by the wrapper
    loss = (out * t["dout"]).sum() + (last.t() * t["dlast"].t()).sum()
    got = torch.autograd.grad(loss, leaves)
    saved = mss.gated_scan_fwd_save(t["x"], t["f"], t["i"], t["rate"], initial_state=t["h0"], seq_lens=t["lens"])[2]
    g = mss.gated_scan_bwd(t["x"], t["f"], t["i"], t["rate"], t["dout"], seq_lens=t["lens"], saved_states=saved,
                           dlast_state=t["dlast"], return_dinitial_state=True)
    for u, n in zip(got, ("dx", "dfgate", "digate", "drate", "dinitial_state")):
        assert torch.equal(u, g[n]), n
    out, _ = mss.GatedScanFunction.apply(leaves[0], t["f"], t["i"], t["rate"])  # some inputs, no state
    got, = torch.autograd.grad(out.sum(), [leaves[0]])
    assert torch.isfinite(got).all()


def test_gradients_against_differences_on_the_gpu(mss):
    """The loss along a random direction of all inputs at +-e, e = 1/64: the difference quotient is off by
    e^2 / 6 of a third derivative (each factor's is of the order of the factor: 4e-5 of the magnitude
    sums) and by the outputs' rounding, (56 + 3 L) u of M through dout, over e."""
    c = inputs(2, 16, 40, "f32", 41, False, True, 0.3, 0.8)
    rng = np.random.default_rng(2)
    way = {n: rng.standard_normal(c[n].shape) for n in ("x", "f", "i", "rate", "h0")}
    way["rate"] *= 0.1

    def loss(e):
        p = dict(c, **{n: (c[n] + e * way[n]).astype(np.float32) for n in way})
        t = upload(p)
        out, last = mss.gated_scan_fwd(t["x"], t["f"], t["i"], t["rate"], initial_state=t["h0"])
        return float((host64(out) * c["dout"]).sum() + (host64(last) * c["dlast"]).sum()), p

    e = 1.0 / 64
    (up, pu), (down, pd) = loss(e), loss(-e)
    t = upload(c)
    g = mss.gated_scan_bwd(t["x"], t["f"], t["i"], t["rate"], t["dout"], initial_state=t["h0"],
                           dlast_state=t["dlast"], return_dinitial_state=True)
    along = sum(float((host64(g[k]) * (pu[n].astype(np.float64) - pd[n])).sum())
                for k, n in (("dx", "x"), ("dfgate", "f"), ("digate", "i"), ("drate", "rate"), ("dinitial_state", "h0")))
    mag = oracle.gated_scan_bwd(np.abs(c["x"]), c["f"], c["i"], c["rate"], np.abs(c["dout"]), np.abs(c["h0"]), None,
                                np.abs(c["dlast"]))
    size = sum(float((mag["m_" + k] * np.abs(way[n])).sum()) for k, n in
               (("dx", "x"), ("dfgate", "f"), ("digate", "i"), ("drate", "rate"), ("dh0", "h0"))) * 2 * e
    M, Ml, _ = oracle.gated_scan(np.abs(c["x"]), c["f"], c["i"], c["rate"], np.abs(c["h0"]))
    noise = (56 + 120) * U * float((M * np.abs(c["dout"])).sum() + (Ml * np.abs(c["dlast"])).sum())
    assert abs(up - down - along) <= 1e-3 * size + 2 * noise, (up - down, along, size, noise)
    assert abs(along) > 4 * (1e-3 * size + 2 * noise)  # the direction says something


@pytest.mark.parametrize("B,D,L,dtype,lens", [(4, 5120, 2048, "bf16", False), (3, 1531, 2041, "f32", True)])
def test_layer_shapes(mss, B, D, L, dtype, lens):
    c = inputs(B, D, L, dtype, 77, lens, lens)
    t = upload(c)
    out, last, saved = mss.gated_scan_fwd_save(t["x"], t["f"], t["i"], t["rate"], initial_state=t["h0"],
                                               seq_lens=t["lens"])
    g = mss.gated_scan_bwd(t["x"], t["f"], t["i"], t["rate"], t["dout"], seq_lens=t["lens"], saved_states=saved,
                           dlast_state=t["dlast"], return_dinitial_state=True)
    ch = slice(None, None, 37)  # the oracle on a thirty-seventh of the channels
    s = dict(c, D=len(range(D)[ch]), **{n: c[n][:, ch] for n in ("x", "f", "i", "dout")}, rate=c["rate"][ch],
             **{n: None if c[n] is None else c[n][:, ch] for n in ("h0", "dlast")})
    what = f"gated layer {B}x{D}x{L} {dtype}"
    check_forward(s, out[:, ch], last[:, ch], saved[:, ch], what)
    check_grads(s, {n: (v[ch] if n == "drate" else v[:, ch]) for n, v in g.items()}, what)


def test_long_context(mss):
    c = inputs(1, 1536, 131072, "f32", 78, False, True)
    t = upload(c)
    out, last, saved = mss.gated_scan_fwd_save(t["x"], t["f"], t["i"], t["rate"], initial_state=t["h0"])
    g = mss.gated_scan_bwd(t["x"], t["f"], t["i"], t["rate"], t["dout"], saved_states=saved,
                           dlast_state=t["dlast"], return_dinitial_state=True)
    ch = [0, 1, 700, 1535]
    s = dict(c, D=4, **{n: c[n][:, ch] for n in ("x", "f", "i", "dout", "h0", "dlast")}, rate=c["rate"][ch])
    check_forward(s, out[:, ch], last[:, ch], saved[:, ch], "gated long context")
    check_grads(s, {n: (v[ch] if n == "drate" else v[:, ch]) for n, v in g.items()}, "gated long context")


@pytest.mark.parametrize("B,D,L", [(4200, 5000, 1), (1, 131, 16400000)])
def test_more_than_2_to_the_31_elements_or_many_rows(mss, B, D, L):
    """21 million rows (beyond any grid's cap), and 2^31 elements in rows of 16.4 million steps: the
    last rows against a call on those rows alone."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    t = [torch.empty((B, D, L), dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(4)]
    rate = torch.rand(D, generator=g, device="cuda") + 0.1
    x, f, i, dout = t
    out, last, saved = mss.gated_scan_fwd_save(x, f, i, rate)
    n = 3
    part = [v[-1:, -n:].contiguous() for v in t]
    o, l, s = mss.gated_scan_fwd_save(*part[:3], rate[-n:].contiguous())
    # the same rows split over the time axis in another way: within the forward's limits of each other
    lim = 3 * (56 + 3 * min(L, 20000)) * U
    scale = float(o.float().abs().max()) * 100 + 1
    assert float((out[-1:, -n:].float() - o.float()).abs().max()) <= lim * scale + 2.0 ** -7 * float(o.float().abs().max())
    assert float((last[-1:, -n:] - l).abs().max()) <= lim * scale
    del out, last
    gr = mss.gated_scan_bwd(x, f, i, rate, dout, saved_states=saved)
    gp = mss.gated_scan_bwd(*part[:3], rate[-n:].contiguous(), part[3], saved_states=s)
    for k in ("dx", "dfgate", "digate"):
        a, b = gr[k][-1:, -n:].float(), gp[k].float()
        assert float((a - b).abs().max()) <= 2 * lim * (float(b.abs().max()) * 100 + 1) + 2.0 ** -7 * float(b.abs().max()), k
    if B > 1:  # every row of a one-step scan by its closed form
        r = rate[:, None] * torch.sigmoid(f.float())
        want = torch.sqrt(-torch.expm1(-2 * r)) * torch.sigmoid(i.float()) * x.float()
        got = mss.gated_scan_fwd(x, f, i, rate, return_last_state=False)
        assert bool(((got.float() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5 * want.abs() + 1e-30).all())


def test_captured_without_a_call_before_and_replayed(mss):
    """Forward, backward and token step captured at once with no warm-up; two graphs of the same calls
    replayed on two streams at the same time, each checked on every replay against eager calls."""
    import torch
    graphs = []
    for k in range(2):
        t = upload(inputs(2, 24, 1500, "bf16", 50 + k, True, True))
        tok = [t[n][..., 0].contiguous() for n in ("x", "f", "i")]
        st = torch.zeros((2, 24), device="cuda")
        torch.cuda.synchronize()

        def body(t=t, tok=tok, st=st):
            out, last, saved = mss.gated_scan_fwd_save(t["x"], t["f"], t["i"], t["rate"], initial_state=t["h0"],
                                                       seq_lens=t["lens"])
            g = mss.gated_scan_bwd(t["x"], t["f"], t["i"], t["rate"], t["dout"], seq_lens=t["lens"],
                                   saved_states=saved, dlast_state=t["dlast"], return_dinitial_state=True)
            st.copy_(last)
            return [out, last, saved, *g.values(), mss.gated_state_update(st, *tok, t["rate"]), st]

        stream = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            res = body()
        graphs.append((t, body, stream, graph, res))
    for rep in range(3):
        want = []
        for k, (t, body, *_r) in enumerate(graphs):
            n = upload(inputs(2, 24, 1500, "bf16", 60 + 2 * rep + k, True, True))
            for name in ("x", "f", "i", "dout", "h0", "dlast", "lens"):
                t[name].copy_(n[name])
            want.append([v.clone() for v in body()])
        torch.cuda.synchronize()
        for _, _, stream, graph, _ in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for k, (_, _, _, _, res) in enumerate(graphs):
            assert all(torch.equal(a, b) for a, b in zip(res, want[k])), (rep, k)


def test_two_streams_at_once(mss):
    import torch
    ts = [upload(inputs(1, 40, 9000, "f32", 80 + k, False, True)) for k in range(2)]
    torch.cuda.synchronize()

    def work(t):
        out, last, saved = mss.gated_scan_fwd_save(t["x"], t["f"], t["i"], t["rate"], initial_state=t["h0"])
        g = mss.gated_scan_bwd(t["x"], t["f"], t["i"], t["rate"], t["dout"], saved_states=saved)
        return [out, last, *g.values()]

    alone = [[v.clone() for v in work(t)] for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    for _ in range(3):
        got = []
        for s, t in zip(streams, ts):
            with torch.cuda.stream(s):
                got.append(work(t))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for u, v in zip(alone, got) for a, b in zip(u, v))
