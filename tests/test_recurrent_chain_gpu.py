"""The new operators as they are used together: a block (conv, gated scan) trained through autograd, and
a small recurrent language model decoded by beam search with its states reordered every token."""
import numpy as np
import pytest

import oracle
from tests.gpu_helpers import dev, host64
from tests.test_gated_gpu import mss  # noqa: F401

pytestmark = pytest.mark.gpu


def test_block_gradients(mss):  # noqa: F811
    """conv -> gated scan (value and both gates from the conv's output by per-channel factors), loss from
    the outputs and both final states; every parameter's gradient against the chain of the fp64
    definitions.  The chain is linear in the outer gradients and its factors are of order 1; each link is off
    by at most (2 (56 + 3 L) + 64) u of its magnitudes (see the operators' own tests), L = 300, three gate
    paths and the conv's 256 u added: 1.5e-4 of the largest gradient with a factor 10 for the magnitudes'
    cancellation."""
    import torch
    rng = np.random.default_rng(0)
    B, D, L, K = 2, 10, 300, 4
    x, dout = (rng.standard_normal((B, D, L)).astype(np.float32) for _ in range(2))
    w, b = (0.5 * rng.standard_normal((D, K))).astype(np.float32), (0.1 * rng.standard_normal(D)).astype(np.float32)
    st, dfin = (rng.standard_normal((B, D, K - 1)).astype(np.float32) for _ in range(2))
    h0, dlast = (rng.standard_normal((B, D)).astype(np.float32) for _ in range(2))
    rate = rng.uniform(0.01, 0.3, D).astype(np.float32)
    cf, ci = (rng.standard_normal((D, 1)).astype(np.float32) for _ in range(2))
    lens = np.array([300, 123], np.int32)

    leaves = {n: dev(v).requires_grad_() for n, v in
              dict(x=x, w=w, b=b, st=st, h0=h0, rate=rate, cf=cf, ci=ci).items()}
    u, fin = mss.CausalConv1dFunction.apply(leaves["x"], leaves["w"], leaves["b"], leaves["st"])
    out, last = mss.GatedScanFunction.apply(u, u * leaves["cf"], u * leaves["ci"], leaves["rate"], leaves["h0"],
                                            torch.from_numpy(lens).cuda())
    loss = (out * dev(dout)).sum() + (last * dev(dlast)).sum() + (fin * dev(dfin)).sum()
    got = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))

    ru, _ = oracle.causal_conv1d(x, w, b, state=st)
    g = oracle.gated_scan_bwd(ru, ru * cf, ru * ci, rate, dout, h0, lens, dlast)
    du = g["dx"] + g["dfgate"] * cf + g["digate"] * ci
    c = oracle.causal_conv1d_bwd(x, w, du, b, st, True, dfin)
    want = dict(x=c["dx"], w=c["dweight"], b=c["dbias"], st=c["dstate"], h0=g["dh0"], rate=g["drate"],
                cf=(g["dfgate"] * ru).sum((0, 2))[:, None], ci=(g["digate"] * ru).sum((0, 2))[:, None])
    for n in leaves:
        r = want[n]
        assert np.abs(host64(got[n]) - r).max() <= 1.5e-4 * 10 * max(1e-3, np.abs(r).max()), n


class Model:
    """A one-layer recurrent language model's weights (fp32) and its fp64 step."""

    def __init__(self, V, D, K, seed):
        rng = np.random.default_rng(seed)
        self.emb = rng.standard_normal((V, D)).astype(np.float32)
        self.w, self.b = (0.5 * rng.standard_normal((D, K))).astype(np.float32), np.zeros(D, np.float32)
        self.wf, self.wi = ((rng.standard_normal((D, D)) / np.sqrt(D)).astype(np.float32) for _ in range(2))
        self.rate = rng.uniform(0.05, 0.5, D).astype(np.float32)
        self.head = (1.5 * rng.standard_normal((D, V))).astype(np.float32)

    def step(self, tokens, win, h):  # tokens (R,), win (R, D, K-1), h (R, D): fp64 logits and new states
        x = self.emb[tokens].astype(np.float64)
        u, win = oracle.causal_conv1d(x[:, :, None], self.w, self.b, state=win)
        u = u[..., 0]
        h = oracle.gated_state_update(h, u, u @ self.wf.astype(np.float64), u @ self.wi.astype(np.float64), self.rate)
        return h @ self.head.astype(np.float64), win, h


def test_beam_search_decodes_the_model(mss):  # noqa: F811
    """Eight tokens of beam search with bound steps (conv, gated scan, selection with reordering), the
    first eager, the rest replayed from one graph, against the same search in fp64: the same parents and
    tokens at every step (scores stand 1e-3 apart or more, fp32 moves them by about 1e-5), the same scores
    and states."""
    import torch
    V, D, K, B, N, end = 300, 32, 4, 3, 4, 5
    m = Model(V, D, K, 4)
    R = B * N
    first = np.repeat(np.arange(10, 10 + B), N)
    rs = np.full((B, N), -np.inf)
    rs[:, 0] = 0.0
    rfin = np.zeros((B, N), np.int64)
    rwin, rh = np.zeros((R, D, K - 1)), np.zeros((R, D))

    tok = torch.from_numpy(first.astype(np.int32)).cuda().view(B, N)
    emb, wf, wi, head = dev(m.emb), dev(m.wf), dev(m.wi), dev(m.head)
    win, h = torch.zeros((R, D, K - 1), device="cuda"), torch.zeros((R, D), device="cuda")
    scores, fin = dev(rs.astype(np.float32)), torch.zeros((B, N), dtype=torch.int32, device="cuda")
    x, f, i, logits = (torch.zeros((R, n), device="cuda") for n in (D, D, D, V))
    stream = torch.cuda.Stream()
    conv = mss.Conv1dUpdateStep(win, x, dev(m.w), dev(m.b), stream=stream)
    scan = mss.GatedUpdateStep(h, conv.out, f, i, dev(m.rate), stream=stream)
    beam = mss.BeamSearchStep(logits.view(B, N, V), scores, [win, h], finished=fin, end_token=end, stream=stream)

    def step():
        torch.index_select(emb, 0, tok.view(-1), out=x)
        u = conv()
        torch.mm(u, wf, out=f)
        torch.mm(u, wi, out=i)
        torch.mm(scan(), head, out=logits)
        beam()
        tok.copy_(beam.tokens)

    torch.cuda.synchronize()
    graph = None
    for t in range(8):
        rl, rwin, rh = m.step(first, rwin, rh)
        full = oracle.beam_select(rl.reshape(B, N, V), rs, k=N + 1, finished=rfin, end_token=end)
        gaps = -np.diff(full[0], axis=1)
        assert gaps[np.isfinite(gaps)].min() > 1e-3, "the seed leaves a near tie"
        rs, rp, rt, rfin = (a[:, :N] for a in full)
        rwin, rh = oracle.beam_reorder(rwin, rp), oracle.beam_reorder(rh, rp)
        first = rt.reshape(-1)
        if t == 0:
            with torch.cuda.stream(stream):
                step()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert beam.parents.cpu().numpy().tolist() == rp.tolist(), t
        assert beam.tokens.cpu().numpy().tolist() == rt.tolist(), t
        assert fin.cpu().numpy().tolist() == rfin.tolist(), t
        # 1e-5 a step in the logits' units (products of 32 fp32 terms of size up to 10: 32 * 10 * 2^-24 =
        # 2e-5), added up in the scores
        assert np.abs(scores.cpu().numpy() - rs)[np.isfinite(rs)].max() < 1e-4 * (t + 1), t
        assert np.abs(host64(h) - rh).max() < 1e-4 and np.abs(host64(win) - rwin).max() < 1e-6, t


def test_two_host_threads(mss):  # noqa: F811
    """Every operator from two host threads at once, each on a stream of its own: nothing is shared, so each
    thread gets what the calls give alone, bit for bit."""
    import threading

    import torch

    def inputs(k):
        g = torch.Generator(device="cuda").manual_seed(k)
        n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        return dict(x=n(2, 70, 1500), f=n(2, 70, 1500), i=n(2, 70, 1500), d=n(2, 70, 1500), rate=n(70).abs() * 0.1 + 0.01,
                    w=n(70, 4), logits=n(3, 5, 4000), scores=n(3, 5), st=n(15, 33, 16),
                    par=torch.randint(0, 5, (3, 5), generator=g, device="cuda", dtype=torch.int32))

    def work(t):
        out, last, saved = mss.gated_scan_fwd_save(t["x"], t["f"], t["i"], t["rate"])
        g = mss.gated_scan_bwd(t["x"], t["f"], t["i"], t["rate"], t["d"], saved_states=saved)
        c = mss.causal_conv1d_bwd(t["x"], t["w"], t["d"])
        sel = mss.beam_select(t["logits"], t["scores"])
        st = mss.beam_reorder([t["st"].clone()], t["par"])[0]
        up = last.clone()
        o = mss.gated_state_update(up, t["x"][..., 0].contiguous(), t["f"][..., 0].contiguous(),
                                   t["i"][..., 0].contiguous(), t["rate"])
        return [out, last, *g.values(), *c.values(), *sel, st, up, o]

    ts = [inputs(k) for k in range(2)]
    want = [[v.clone() for v in work(t)] for t in ts]
    torch.cuda.synchronize()
    wrong = []

    def run(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got = work(ts[k])
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[k])):
                        wrong.append(k)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # an assertion in a thread would be lost
            wrong.append(repr(e))

    threads = [threading.Thread(target=run, args=(k,)) for k in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong, wrong
