"""fp64 definitions of the gated scan, the causal conv's gradients and beam search's selection.

Written step by step in numpy float64 from the formulas, sequential in time and vectorised over
the independent rows.  Test infrastructure only, like the rest of this package.
"""
from __future__ import annotations

import numpy as np


def _f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def _sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def _lens(seq_lens, batch, L):
    if seq_lens is None:
        return np.full(batch, L)
    return np.clip(np.asarray(seq_lens, dtype=np.int64), 0, L)


def _gates(x, fgate, igate, rate):
    """a, the input term v, m = sqrt(1 - a^2), sigmoid(fgate), sigmoid(igate); rate broadcastable."""
    r, p = _sigmoid(fgate), _sigmoid(igate)
    s = rate * r
    m = np.sqrt(-np.expm1(-2.0 * s))
    return np.exp(-s), m * p * x, m, r, p


def gated_scan(x, fgate, igate, rate, h0=None, seq_lens=None):
    """out (batch, d_inner, L), last state (batch, d_inner) and the state entering every step
    (batch, d_inner, L) of the gated scan."""
    x, fgate, igate, rate = _f64(x), _f64(fgate), _f64(igate), _f64(rate)
    B, D, L = x.shape
    lens = _lens(seq_lens, B, L)
    a, v, _, _, _ = _gates(x, fgate, igate, rate[:, None])
    h = np.zeros((B, D)) if h0 is None else _f64(h0).copy()
    out, before = np.zeros((B, D, L)), np.empty((B, D, L))
    for t in range(L):
        before[..., t] = h
        on = (t < lens)[:, None]
        h = np.where(on, a[..., t] * h + v[..., t], h)
        out[..., t] = np.where(on, h, 0.0)
    return out, h, before


def gated_scan_bwd(x, fgate, igate, rate, dout, h0=None, seq_lens=None, dlast=None):
    """Gradients of sum(dout * out) + sum(dlast * last_state): a dict of dx, dfgate, digate
    (batch, d_inner, L), drate (d_inner,) and dh0 (batch, d_inner), and under "m_" + name the same
    sums with every term's magnitude (what the rounding of a sum is relative to)."""
    x, fgate, igate, rate, dout = _f64(x), _f64(fgate), _f64(igate), _f64(rate), _f64(dout)
    B, D, L = x.shape
    lens = _lens(seq_lens, B, L)
    _, _, before = gated_scan(x, fgate, igate, rate, h0, seq_lens)
    a, _, m, r, p = _gates(x, fgate, igate, rate[:, None])
    with np.errstate(divide="ignore", invalid="ignore"):
        dm = np.where(m > 0, a * a / m, 0.0)  # d m / d s, s = rate r
    g = {n: np.zeros((B, D, L)) for n in ("dx", "dfgate", "digate", "m_dx", "m_dfgate", "m_digate")}
    drate, m_drate = np.zeros((B, D)), np.zeros((B, D))
    w = np.zeros((B, D)) if dlast is None else _f64(dlast).copy()
    mw = np.abs(w)
    for t in range(L - 1, -1, -1):
        on = (t < lens)[:, None]
        at, G, M = a[..., t], dout[..., t] + w, np.abs(dout[..., t]) + mw
        into = dm[..., t] * p[..., t] * x[..., t]
        ds = G * (into - at * before[..., t])
        mds = M * (np.abs(into) + at * np.abs(before[..., t]))
        r1, s = r[..., t], rate * r[..., t]
        dv, q = m[..., t] * p[..., t], p[..., t] * (1 - p[..., t])
        for n, val in (("dx", G * dv), ("dfgate", ds * s * (1 - r1)), ("digate", G * m[..., t] * x[..., t] * q),
                       ("m_dx", M * dv), ("m_dfgate", mds * s * (1 - r1)),
                       ("m_digate", M * m[..., t] * np.abs(x[..., t]) * q)):
            g[n][..., t] = np.where(on, val, 0.0)
        drate += np.where(on, ds * r1, 0.0)
        m_drate += np.where(on, mds * r1, 0.0)
        w, mw = np.where(on, at * G, w), np.where(on, at * M, mw)
    g.update(drate=drate.sum(0), m_drate=m_drate.sum(0), dh0=w, m_dh0=mw)
    return g


def gated_state_update(state, x, fgate, igate, rate):
    """One step from `state` (batch, d_inner): the new state, which is also the output."""
    a, v, _, _, _ = _gates(_f64(x), _f64(fgate), _f64(igate), _f64(rate))
    return a * _f64(state) + v


def causal_conv1d_bwd(x, weight, dout, bias=None, state=None, silu=True, dfinal=None):
    """Gradients of sum(dout * out) + sum(dfinal * final_state) of the causal conv: a dict of dx,
    dweight, dbias and dstate, and "m_" + name with every term's magnitude."""
    x, w, dout = _f64(x), _f64(weight), _f64(dout)
    B, D, L = x.shape
    K = w.shape[1]
    win = np.concatenate([np.zeros((B, D, K - 1)) if state is None else _f64(state), x], -1)
    y = np.zeros((B, D, L)) + (0.0 if bias is None else _f64(bias)[:, None])
    for k in range(K):
        y = y + w[:, k, None] * win[..., k:k + L]
    sg = _sigmoid(y)
    d = dout * (sg * (1 + y * (1 - sg))) if silu else dout
    dwin, mwin = np.zeros_like(win), np.zeros_like(win)
    dw, mw = np.zeros((D, K)), np.zeros((D, K))
    for k in range(K):
        dwin[..., k:k + L] += w[:, k, None] * d
        mwin[..., k:k + L] += np.abs(w[:, k, None] * d)
        dw[:, k] = (d * win[..., k:k + L]).sum((0, 2))
        mw[:, k] = np.abs(d * win[..., k:k + L]).sum((0, 2))
    if dfinal is not None and K > 1:
        dwin[..., L:] += _f64(dfinal)
        mwin[..., L:] += np.abs(_f64(dfinal))
    return dict(dx=dwin[..., K - 1:], dweight=dw, dbias=d.sum((0, 2)), dstate=dwin[..., :K - 1],
                m_dx=mwin[..., K - 1:], m_dweight=mw, m_dbias=np.abs(d).sum((0, 2)), m_dstate=mwin[..., :K - 1])


def beam_select(logits, scores, k=None, finished=None, end_token=None):
    """The k best continuations of every request: (scores, parents, tokens, finished), each
    (batch, k).

    A live beam's continuation by token v scores score + logit_v - log sum exp(logits); a finished
    beam has one, by end_token at its own score.  Continuations whose score is -inf or not a number
    do not exist (a NaN logit counts as -inf).  Order: higher score first; equal scores by beam,
    within a beam by higher logit, then by token.  Missing ones: (-inf, 0, 0, 0)."""
    x, sc = _f64(logits), _f64(scores)
    B, N, V = x.shape
    k = N if k is None else k
    x = np.where(np.isnan(x), -np.inf, x)
    out = (np.full((B, k), -np.inf), np.zeros((B, k), np.int64), np.zeros((B, k), np.int64),
           np.zeros((B, k), np.int64))
    for b in range(B):
        found = []
        for i in range(N):
            if finished is not None and finished[b, i]:
                if sc[b, i] > -np.inf:
                    found.append((-sc[b, i], i, 0, int(end_token), 1))
                continue
            top = x[b, i].max() if V else -np.inf
            if not np.isfinite(top):
                continue
            lse = top + np.log(np.exp(x[b, i] - top).sum())
            order = np.argsort(-x[b, i], kind="stable")[:k]
            for rank, v in enumerate(order):
                s = sc[b, i] + (x[b, i, v] - lse)
                if s > -np.inf:
                    found.append((-s, i, rank, int(v), 0))
        for j, (s, i, _, v, done) in enumerate(sorted(found)[:k]):
            out[0][b, j], out[1][b, j], out[2][b, j] = -s, i, v
            out[3][b, j] = 1 if done or (end_token is not None and v == end_token) else 0
    return out


def beam_reorder(state, parents):
    """state (batch * beams, ...) with row b * beams + j taken from row b * beams + parents[b, j];
    a parent outside [0, beams) leaves the row as it is."""
    state, parents = np.asarray(state), np.asarray(parents)
    B, N = parents.shape
    own = np.arange(N)[None, :]
    p = np.where((parents >= 0) & (parents < N), parents, own) + N * np.arange(B)[:, None]
    return state[p.reshape(-1)]
