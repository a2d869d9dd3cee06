"""GPU tests of the gated scan's long rows (several waves to a row, rows cut into segments, rates on both
sides of 1/4) whose limits follow the memory that the gates leave, not the length.

u = 2^-24.  Errors are carried step by step beside the values, first order, and the whole taken 1.02 times
for the products of errors (every relative error here is below 1%):
  - sigmoid(f): e^-f carries the rounding of f log2 e, |f| u, and 8 u of exp2, 1 + e and the reciprocal;
    1 - sigmoid the same; s = rate r two roundings more: es = (|f| + 10) u.
  - a = e^-s: s (es + 2 u) for the exponent, 2 u for exp2:  ea.
  - q = 1 - a^2: es through y = 2 s (d log q / d log y <= 1) and 6 u for the polynomial and its fit; above
    y = 1/2 instead 2 a^2 ea / q and u / q.  m = sqrt(q), or its reciprocal: half of that and 2 u:  em.
  - the input term v = m p x: em, p's and 4 u:  ev.
  - the state: E_t = a_t (E_{t-1} + (ea + 3 u) M_{t-1}) + (ev + 3 u) |v_t| with M the sums of magnitudes: one
    rounding for the product of the decays, one for the multiply-add and one for its place in a fold.  A
    term passes through at most 6 joins of lanes, 8 of waves, 6 of segments and 12 steps of a lane's second
    walk more: 32 u M.
  - the adjoint the same with dout for the input term, which is exact.
  - a product of such factors: each one's error times the others' values.  ds = G (X1 - X2) with X1 = a^2 / m p x
    (2 ea + em + ep + 6 u) and X2 = a h.
  - drate sums B L such terms: each one's error, and the roundings of the sum, at most L / 64 + B + 32 in a row,
    each u of the sum of magnitudes.
  - a bf16 result adds half a step, 2^-8 of its value.

Every test asserts that the limits are worth something: with inputs of one sign zeros fail for every element
(for nearly all of dfgate's, whose terms differ in sign), drate stands ten times above its limit, and nearly
every piece of a row adds more to it than that limit; with inputs of both signs zeros fail for nearly all
elements."""
import numpy as np
import pytest

from synth import round_to_bf16
from tests.gpu_helpers import dev, host64
from tests.test_gated_gpu import check, mss  # noqa: F401

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def make(B, D, L, dtype, seed, sign, lens=False, lo=0.004, hi=1.5):
    """Rates spread over their logarithm, on both sides of 1/4."""
    rng = np.random.default_rng(9000 + seed)
    rnd = round_to_bf16 if dtype == "bf16" else (lambda a: a)
    c = dict(B=B, D=D, L=L, dtype=dtype)
    for n in ("f", "i"):
        c[n] = rnd(np.clip(rng.standard_normal((B, D, L)), -6, 6).astype(np.float32))
    for n in ("x", "dout"):
        v = rng.uniform(0.5, 1.5, (B, D, L)) if sign else rng.standard_normal((B, D, L))
        c[n] = rnd(v.astype(np.float32))
    c["rate"] = np.exp(rng.uniform(np.log(lo), np.log(hi), D)).astype(np.float32)
    c["rate"][:2] = (lo, hi)[:D]
    c["h0"], c["dlast"] = (rng.uniform(0.5, 1.5, (B, D)).astype(np.float32) for _ in range(2))
    c["lens"] = None
    if lens:
        c["lens"] = rng.integers(L // 2, L + 1, B).astype(np.int32)
        c["lens"][-1] = L
    return c


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def recur(a, b, y):
    """y_t = a_t y_{t-1} + b_t along the last axis from y (rows,): all blocks of the axis at once from zero, then
    the blocks in order, each from the end of the one before (in fp64 the order does not matter here)."""
    R, L = a.shape
    T = 256
    C = -(-L // T)
    aa, bb = np.ones((R, C * T)), np.zeros((R, C * T))
    aa[:, :L], bb[:, :L] = a, b
    aa, bb = (np.ascontiguousarray(v.reshape(R, C, T).transpose(2, 0, 1)) for v in (aa, bb))  # (T, R, C)
    for t in range(1, T):
        bb[t] += aa[t] * bb[t - 1]
        aa[t] *= aa[t - 1]
    first = np.empty((R, C))  # what enters each block
    for k in range(C):
        first[:, k] = y
        y = aa[-1, :, k] * y + bb[-1, :, k]
    return (bb + aa * first).transpose(1, 2, 0).reshape(R, C * T)[:, :L]


def carried(c, cuts=None):
    """{name: (value, limit)} of every output and gradient, and drate's parts per row and piece of `cuts`
    steps (B, D, pieces)."""
    B, D, L = c["x"].shape
    x, f, i, dout = (c[n].astype(np.float64).reshape(B * D, L) for n in ("x", "f", "i", "dout"))
    h0, dlast = (c[n].astype(np.float64).reshape(-1) for n in ("h0", "dlast"))
    rate = np.tile(c["rate"].astype(np.float64), B)[:, None]
    lens = np.full(B, L) if c["lens"] is None else c["lens"]
    on = np.arange(L)[None] < np.repeat(lens, D)[:, None]
    zero = np.zeros((B * D, 1))

    def before(v, first):
        return np.concatenate([first[:, None], v[:, :-1]], 1)

    r, p = sigmoid(f), sigmoid(i)
    s = rate * r
    a = np.exp(-s)
    q = -np.expm1(-2 * s)
    m = np.sqrt(q)
    es, ep = (np.abs(f) + 10) * U, (np.abs(i) + 8) * U
    ea = s * (es + 2 * U) + 2 * U
    eq = np.where(s < 0.249, es + 6 * U, np.maximum(es + 6 * U, (2 * a * a * ea + U) / q))
    em = 0.5 * eq + 2 * U
    ev = em + ep + 4 * U
    v = np.where(on, m * p * x, 0.0)
    step = np.where(on, a, 1.0)  # past a sequence's end nothing moves
    h = recur(step, v, h0)
    M = recur(step, np.abs(v), np.abs(h0))
    M1 = before(M, np.abs(h0))
    E = recur(step, np.where(on, a * (ea + 3 * U) * M1 + (ev + 3 * U) * np.abs(v), 0.0), zero[:, 0])
    h1, E1 = before(h, h0), before(E, zero[:, 0]) + 32 * U * M1
    E = E + 32 * U * M
    # the adjoint, from the end: w_t = a_t (dout_t + w_{t+1}), G_t = dout_t + w_{t+1}
    back = np.where(on, dout, 0.0)[:, ::-1]
    sb = step[:, ::-1]
    w = recur(sb, sb * back, dlast)
    MW = recur(sb, sb * np.abs(back), np.abs(dlast))
    w1, MW1 = before(w, dlast), before(MW, np.abs(dlast))
    MG = np.abs(back) + MW1
    EW = recur(sb, np.where(on[:, ::-1], sb * (U + (ea + 3 * U)[:, ::-1]) * MG, 0.0), zero[:, 0])
    G, EG = back + w1, before(EW, zero[:, 0]) + 33 * U * MG
    G, EG = G[:, ::-1], EG[:, ::-1]
    X1, X2 = a * a / m * p * x, a * h1
    X = X1 - X2
    eX = (2 * ea + em + ep + 6 * U) * np.abs(X1) + a * E1 + (ea + 2 * U) * np.abs(X2) + 2 * U * np.abs(X)
    ds = G * X
    eds = np.abs(G) * eX + EG * (np.abs(X) + eX) + 2 * U * np.abs(ds)
    fac = s * (1 - r)
    res = dict(
        out=(np.where(on, h, 0.0), E), last=(h[:, -1], E[:, -1]), saved=(h1[:, ::512], E1[:, ::512]),
        dx=(G * m * p, m * p * (EG + ev * np.abs(G))),
        digate=(G * m * p * x * (1 - p), np.abs(m * p * x * (1 - p)) * (EG + (ev + ep + 5 * U) * np.abs(G))),
        dfgate=(ds * fac, fac * (eds + (2 * es + 6 * U) * np.abs(ds))),
        dh0=(w[:, -1], EW[:, -1] + 32 * U * MW[:, -1]))
    val, err = np.where(on, ds * r, 0.0), np.where(on, r * (eds + (es + 2 * U) * np.abs(ds)), 0.0)
    for n in ("out", "dx", "digate", "dfgate"):
        res[n] = tuple(np.where(on, k, 0.0) for k in res[n])
    res = {n: tuple(k.reshape(B, D, *k.shape[1:]) for k in e) for n, e in res.items()}
    val, err = val.reshape(B, D, L), err.reshape(B, D, L)
    adds = L / 64 + B + 32
    res["drate"] = (val.sum((0, 2)), err.sum((0, 2)) + adds * U * np.abs(val).sum((0, 2)))
    lim = {}
    for n, (ref, e) in res.items():
        bf = c["dtype"] == "bf16" and n in ("out", "dx", "dfgate", "digate")
        lim[n] = (ref, 1.02 * e + (2.0 ** -8 * np.abs(ref) if bf else 0.0) + 1e-30)
    return lim, np.add.reduceat(val, np.arange(0, L, cuts), axis=2) if cuts else None


def worth(c, lim, parts):
    """What the limits would let through: with inputs of one sign zeros fail for every element (dfgate, whose
    terms differ in sign, and inputs of both signs: for nearly all)."""
    for n, (ref, l) in lim.items():
        live = np.ones(ref.shape, bool)
        if c["lens"] is not None and n in ("out", "dx", "digate", "dfgate"):
            live[:] = np.arange(c["L"]) < c["lens"][:, None, None]
        zeros = ((np.abs(ref) <= l) & live).sum() / live.sum()
        if n == "drate":
            assert not c["sign"] or np.all(np.abs(ref) > 10 * l), (n, float((l / np.abs(ref)).max()))
        else:
            assert zeros <= (0.05 if n == "dfgate" or not c["sign"] else 0.0), (n, zeros)
    if c["sign"]:
        live = np.abs(parts)
        if c["lens"] is not None:  # pieces past a sequence's end add nothing
            live = live[:, :, :int(np.min(c["lens"])) // c["cuts"]]
        kept = live > lim["drate"][1][:, None]
        assert kept.mean() > 0.99, ("a piece of drate could be lost", kept.mean())


# What the rules for waves and segments make of these sizes: rows up to 128 of 128 tiles or more are cut into
# segments; up to 2048 rows of 64 tiles or more take eight waves; then four; then one (more than 1024 rows).
CASES = [
    # B, D, L, dtype, lengths, cuts: steps of the shortest piece whose loss must show
    (1, 3, 70001, "f32", False, 2048),     # segments, rows that are no whole vectors
    (2, 20, 66048, "bf16", True, 6144),    # segments, two rows to a channel
    (1, 128, 65536, "f32", False, 16384),  # segments, four to a row
    (1, 130, 33001, "f32", False, 4096),   # eight waves, one row to a channel
    (2, 130, 33024, "bf16", True, 4096),   # eight waves, parts of drate
    (4, 6, 5001, "bf16", True, 512),       # four waves
    (5, 300, 2048, "bf16", False, 512),    # one wave, parts of drate
    (4, 300, 2043, "f32", True, 512),      # one wave, a block adds the rows up
]


@pytest.mark.parametrize("B,D,L,dtype,lens,cuts", CASES)
@pytest.mark.parametrize("sign", [True, False])
def test_within_the_gates_memory(mss, B, D, L, dtype, lens, cuts, sign):  # noqa: F811
    c = dict(make(B, D, L, dtype, B + D + L, sign, lens), sign=sign, cuts=cuts)
    lim, parts = carried(c, cuts)
    worth(c, lim, parts)
    import torch
    t = {n: dev(c[n], dtype) for n in ("x", "f", "i", "dout")}
    t.update({n: dev(c[n]) for n in ("rate", "h0", "dlast")})
    seq = None if c["lens"] is None else torch.from_numpy(c["lens"]).cuda()
    out, last, saved = mss.gated_scan_fwd_save(t["x"], t["f"], t["i"], t["rate"], initial_state=t["h0"], seq_lens=seq)
    g = mss.gated_scan_bwd(t["x"], t["f"], t["i"], t["rate"], t["dout"], seq_lens=seq, saved_states=saved,
                           dlast_state=t["dlast"], return_dinitial_state=True)
    got = dict(out=out, last=last, saved=saved, dx=g["dx"], dfgate=g["dfgate"], digate=g["digate"],
               dh0=g["dinitial_state"], drate=g["drate"])
    for n, (ref, l) in lim.items():
        check(got[n], ref, l, f"{B}x{D}x{L} {dtype} {n}")


def test_rows_of_16_million_steps(mss):  # noqa: F811
    """1 x 131 x 16400000 (2^31 elements and more): out and the gradients in windows at a row's start, where
    the row crosses 2^31 elements, and at its end, against the fp64 definition run on the window alone.  Rates of
    0.3 to 1 and gates about sigmoid(0) leave in 12000 steps on either side, each decaying by e^-0.15 in the
    mean, e^-1800 of what lies outside: the window's middle does not depend on it.  drate
    (inputs of one sign) against the sum of ds r that the gradients give: df = ds s (1 - r), so ds r =
    df / (rate (1 - r))."""
    import torch
    D, L, edge = 131, 16400000, 12000
    g = torch.Generator(device="cuda").manual_seed(3)
    f, i = (torch.empty((1, D, L), dtype=torch.bfloat16, device="cuda").normal_(generator=g).clamp_(-4, 4)
            for _ in range(2))
    x, dout = (torch.empty((1, D, L), dtype=torch.bfloat16, device="cuda").uniform_(0.5, 1.5, generator=g)
               for _ in range(2))
    rate = torch.rand(D, generator=g, device="cuda") * 0.7 + 0.3
    rate[-1] = 0.3
    out, last, saved = mss.gated_scan_fwd_save(x, f, i, rate)
    gr = mss.gated_scan_bwd(x, f, i, rate, dout, saved_states=saved, return_dinitial_state=True)
    at31 = 2 ** 31 - (D - 1) * L  # the last row's step that is element 2^31
    assert edge < at31 < L - edge
    for lo, keep_lo, keep_hi, hi in ((0, 0, 600, 600 + edge), (at31 - edge, at31 - 600, at31 + 600, at31 + edge),
                                     (L - edge - 600, L - 600, L, L)):
        w = {n: v[:, -2:, lo:hi].float().cpu().numpy() for n, v in (("x", x), ("f", f), ("i", i), ("dout", dout))}
        c = dict(w, B=1, D=2, L=hi - lo, dtype="bf16", sign=True, rate=rate[-2:].cpu().numpy(),
                 h0=np.zeros((1, 2), np.float32), dlast=np.zeros((1, 2), np.float32), lens=None)
        lim, _ = carried(c)
        k = slice(keep_lo - lo, keep_hi - lo)
        for n, v in (("out", out), ("dx", gr["dx"]), ("dfgate", gr["dfgate"]), ("digate", gr["digate"])):
            ref, l = (z[..., k] for z in lim[n])
            assert (np.abs(ref) <= l).mean() < 0.02, n
            check(v[:, -2:, keep_lo:keep_hi], ref, l, f"16.4M steps {n} at {keep_lo}")
        if hi == L:
            check(last[:, -2:], *lim["last"], "16.4M steps last")
        if lo == 0:
            check(gr["dinitial_state"][:, -2:], *lim["dh0"], "16.4M steps dh0")
    # the elements of df are off by their own errors and half a bf16 step, 2^-8; the kernel's sum over eight waves
    # of 64 lanes by L / 512 + 64 additions in a row
    for d in (D - 2, D - 1):
        r = torch.sigmoid(f[0, d].double())
        terms = gr["dfgate"][0, d].double() / (float(rate[d]) * (1 - r))
        total, size = float(terms.sum()), float(terms.abs().sum())
        # per term three times the state's and the adjoint's relative error, 5 u for each step of a memory of at
        # most 40 (1 / 0.3 where the gates stand at 1/2; a run of shut gates is short), and 256 u
        tol = size * (2.0 ** -8 + (3 * 5 * 40 + 256) * U + (L / 512 + 64) * U)
        assert abs(float(gr["drate"][d]) - total) <= tol, (d, float(gr["drate"][d]), total, tol)
        assert abs(total) > 20 * tol
