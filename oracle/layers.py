"""fp64 definitions of the RMS norm, linear attention with a decay per head, and token log probabilities.

Written step by step in numpy float64 from the formulas.  Test infrastructure only, like the rest of this package.
Functions that take `magnitude` give the same sums with every term's magnitude, what the rounding of a sum is relative to.
"""
from __future__ import annotations

import numpy as np

from .recurrent import _f64, _lens


def rms_norm(z, weight, eps):
    """out and rstd of rows z (R, W)."""
    z, weight = _f64(z), _f64(weight)
    rstd = 1.0 / np.sqrt(np.mean(z * z, -1) + eps)
    return z * rstd[:, None] * weight, rstd


def rms_norm_bwd(z, weight, eps, dout, dstream=None):
    """dz and dweight, and under "m_" + name their magnitudes."""
    z, weight, dout = _f64(z), _f64(weight), _f64(dout)
    _, r = rms_norm(z, weight, eps)
    zh, wd = z * r[:, None], weight * dout
    add = 0.0 if dstream is None else _f64(dstream)
    return {"dz": r[:, None] * (wd - zh * np.mean(wd * zh, -1, keepdims=True)) + add,
            "m_dz": r[:, None] * (np.abs(wd) + np.abs(zh) * np.mean(np.abs(wd * zh), -1, keepdims=True)) + np.abs(add),
            "dweight": np.sum(dout * zh, 0), "m_dweight": np.sum(np.abs(dout * zh), 0)}


def _wide(t, heads):
    """(B, L, shared heads, d) -> (B, L, heads, d)"""
    return np.repeat(_f64(t), heads // t.shape[2], axis=2)


def _walk(q, k, v, decay, S, lens):
    """Outputs (B, L, H, dv) of S_t = decay S_{t-1} + k_t v_t^T seen by q_t, and the state after."""
    B, L, H, _ = q.shape
    out, S = np.zeros((B, L, H, v.shape[-1])), S.copy()
    for t in range(L):
        on = (t < lens)[:, None, None, None]
        new = decay[:, None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        S = np.where(on, new, S)
        out[:, t] = np.where(on[..., 0], np.einsum("bhk,bhkv->bhv", q[:, t], S), 0.0)
    return out, S


def linear_attention(q, k, v, rate, scale, S0=None, seq_lens=None, magnitude=False):
    """out (B, L, H, V) and the last state (B, H, K, V)."""
    H = len(rate)
    q, k, v = (_wide(t, H) for t in (q, k, v))
    if magnitude:
        q, k, v = np.abs(q), np.abs(k), np.abs(v)
    S = np.zeros((q.shape[0], H, q.shape[-1], v.shape[-1])) if S0 is None else _f64(S0)
    out, S = _walk(q, k, v, np.exp(-_f64(rate)), np.abs(S) if magnitude else S, _lens(seq_lens, q.shape[0], q.shape[1]))
    return scale * out, S


def linear_attention_bwd(q, k, v, rate, scale, dout, S0=None, seq_lens=None, dlast=None, magnitude=False):
    """dq, dk, dv (shared heads summed) and dS0 of sum(dout * out) + sum(dlast * last): the adjoint
    G_t = dS_t: G_t = decay G_{t+1} + scale q_t dout_t^T, G = dlast behind a sequence's last step."""
    H, shared = len(rate), {"dq": q.shape[2], "dk": k.shape[2], "dv": v.shape[2]}
    q, k, v, d = (_wide(t, H) for t in (q, k, v, dout))
    B, L, _, K = q.shape
    V = v.shape[-1]
    S0 = np.zeros((B, H, K, V)) if S0 is None else _f64(S0)
    E = np.zeros((B, H, K, V)) if dlast is None else _f64(dlast)
    if magnitude:
        q, k, v, d, S0, E = (np.abs(t) for t in (q, k, v, d, S0, E))
    lens, decay = _lens(seq_lens, B, L), np.exp(-_f64(rate))
    g = {"dq": scale * _walk(d, v, k, decay, np.swapaxes(S0, -1, -2), lens)[0],
         "dk": np.zeros((B, L, H, K)), "dv": np.zeros((B, L, H, V))}
    G = E.copy()  # the adjoint of the state after step t, before that step's own output
    for t in range(L - 1, -1, -1):
        on = (t < lens)[:, None, None, None]
        now = G + scale * q[:, t, :, :, None] * d[:, t, :, None, :]
        g["dk"][:, t] = np.where(on[..., 0], np.einsum("bhkv,bhv->bhk", now, v[:, t]), 0.0)
        g["dv"][:, t] = np.where(on[..., 0], np.einsum("bhkv,bhk->bhv", now, k[:, t]), 0.0)
        G = np.where(on, decay[:, None, None] * now, G)
    for n, heads in shared.items():
        g[n] = g[n].reshape(B, L, heads, H // heads, -1).sum(3)
    g["dS0"] = G
    return g


def token_logprobs(logits, tokens, top=0):
    """A dict of logprobs, entropy (R,), top_logprobs and top_tokens (R, top), p and logp (R, V).  Rows of -inf alone have
    logprobs -inf, entropy 0 and no alternatives; rows with NaN or +inf are NaN."""
    x = _f64(logits)
    R, V = x.shape
    with np.errstate(invalid="ignore", divide="ignore"):
        m = np.max(x, -1, keepdims=True)
        dead = np.all(x == -np.inf, -1)
        e = np.where(dead[:, None], 0.0, np.exp(x - m))
        s = e.sum(-1, keepdims=True)
        logp = np.where(dead[:, None], -np.inf, x - m - np.log(s))
        p = np.where(dead[:, None], 0.0, e / s)
        entropy = -np.sum(np.where(p > 0, p * logp, p), -1)
    entropy[dead] = 0.0
    ok = (tokens >= 0) & (tokens < V)
    lp = np.where(ok, logp[np.arange(R), np.where(ok, tokens, 0)], 0.0)
    got = {"logprobs": lp, "entropy": entropy, "p": p, "logp": logp}
    if top:
        at = np.argsort(-np.where(np.isnan(x), -np.inf, x), axis=-1, kind="stable")[:, :top]
        tl, tx = np.take_along_axis(logp, at, -1), np.take_along_axis(x, at, -1)
        none = (tx == -np.inf) | np.isnan(tx)
        got["top_logprobs"] = np.full((R, top), -np.inf)
        got["top_tokens"] = np.full((R, top), -1)
        got["top_logprobs"][:, :at.shape[1]] = np.where(none, -np.inf, tl)
        got["top_tokens"][:, :at.shape[1]] = np.where(none, -1, at)
    return got


def token_logprobs_bwd(logits, tokens, g, h=None):
    """dlogits of sum(g * logprobs) + sum(h * entropy), and its terms' magnitude."""
    o = token_logprobs(logits, tokens)
    R, V = np.shape(logits)
    p, ok = o["p"], (tokens >= 0) & (tokens < V)
    dead = np.all(_f64(logits) == -np.inf, -1)
    g = np.where(ok & ~dead, _f64(g), 0.0)[:, None]
    h = np.zeros((R, 1)) if h is None else np.where(dead, 0.0, _f64(h))[:, None]
    with np.errstate(invalid="ignore"):
        logp = np.where(p > 0, o["logp"], 0.0)
    H = o["entropy"][:, None]
    one = np.zeros((R, V))
    one[np.arange(R), np.where(ok, tokens, 0)] = ok
    return g * (one - p) - h * p * (logp + H), np.abs(g) * (one + p) + np.abs(h) * p * (np.abs(logp) + np.abs(H))
