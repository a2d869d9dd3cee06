"""Measured cases of the RMS norm with the residual's addition, linear attention with a decay for each head, and log
probabilities of given tokens.

Each case is one call (or, for the training cases, a forward with its backward) of an operator on synthetic data: `run`
computes it in its plain form from elementary torch operations (`own` false) or through the library (`own` true), `exact`
from the definition in 64 bits.

norm       z = x + residual, in the residual stream's type; out = z / sqrt(mean z^2 + eps) * weight; in 8 bits:
           out / scale in e4m3 with scale = max |out| / 448 over a row, or over each 128 columns of it
attention  S_t = exp(-rate) S_{t-1} + k_t v_t^T, out_t = scale S_t^T q_t, per (batch, head); steps past a sequence's
           length leave the state alone and give 0; q, k and v may each have fewer heads, which neighbours share
logprobs   of given tokens under softmax(logits), the entropy of each row, and its most probable tokens
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


def listed():
    return [
        # one token for one request at the 2.8B width, the residual stream in 32 bits: latency
        {"name": "norm one bf16", "op": "norm", "rows": 1, "width": 2560, "dtype": "bf16", "residual": "f32", "group": -1},
        # prefill of one block of the 2.8B shape, four prompts of 2048
        {"name": "norm layer bf16", "op": "norm", "rows": 8192, "width": 2560, "dtype": "bf16", "residual": "f32",
         "group": -1},
        # the same in front of an 8-bit product, a scale for each row
        {"name": "norm layer 8 bits", "op": "norm", "rows": 4096, "width": 5120, "dtype": "bf16", "residual": "bf16",
         "group": 0},
        # a training step's norm on rows that are no whole vectors
        {"name": "norm train f32", "op": "norm train", "rows": 6123, "width": 2049, "dtype": "f32", "residual": "f32"},
        # prefill of one layer: four full prompts, 32 heads of 128
        {"name": "attention layer bf16", "op": "attention", "batch": 4, "L": 2048, "heads": 32, "q_heads": 32,
         "k_heads": 32, "v_heads": 32, "key_dim": 128, "value_dim": 128, "dtype": "bf16", "lens": False, "h0": False},
        # one long document appended to a kept state, keys and values shared by four heads each
        {"name": "attention long f32", "op": "attention", "batch": 1, "L": 32768, "heads": 16, "q_heads": 16,
         "k_heads": 4, "v_heads": 4, "key_dim": 64, "value_dim": 64, "dtype": "f32", "lens": False, "h0": True},
        # a training step of the Mamba-2 2.7B shape: 80 heads of 64, queries and keys shared by ten heads each
        {"name": "attention train bf16", "op": "attention train", "batch": 4, "L": 2048, "heads": 80, "q_heads": 8,
         "k_heads": 8, "v_heads": 80, "key_dim": 128, "value_dim": 64, "dtype": "bf16", "lens": False, "h0": False},
        # a training step on a batch of different lengths, from carried states
        {"name": "attention train ragged f32", "op": "attention train", "batch": 3, "L": 1531, "heads": 12,
         "q_heads": 12, "k_heads": 12, "v_heads": 12, "key_dim": 64, "value_dim": 96, "dtype": "f32", "lens": True,
         "h0": True},
        # one token for a batch of 64 requests of the 2.7B shape
        {"name": "attention step bf16", "op": "attention step", "batch": 64, "heads": 80, "q_heads": 8, "k_heads": 8,
         "v_heads": 80, "key_dim": 128, "value_dim": 64, "dtype": "bf16"},
        # the logits of one token of one request, with its 20 most probable alternatives: latency
        {"name": "logprobs one f32", "op": "logprobs", "rows": 1, "vocab": 50277, "dtype": "f32", "top": 20,
         "masked": False},
        # a decode step of 128 requests over a large odd vocabulary, part of it masked by a grammar
        {"name": "logprobs batch bf16", "op": "logprobs", "rows": 128, "vocab": 128007, "dtype": "bf16", "top": 5,
         "masked": True},
        # the loss of a training step: 4096 tokens, gradients of the log probabilities and of the entropy
        {"name": "logprobs train bf16", "op": "logprobs train", "rows": 4096, "vocab": 50280, "dtype": "bf16",
         "masked": False},
    ]


def _log_int(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm train", "attention", "attention train", "attention step", "logprobs",
                     "logprobs train"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("norm", "norm train"):
        width = _log_int(rng, 64, 16384)
        if rng.random() < 0.6:
            width = -(-width // 8) * 8
        rows = _log_int(rng, 1, min(65536, (12 << 20 if op == "norm train" else 20 << 20) // width))
        case = {"op": op, "rows": rows, "width": width, "dtype": dtype,
                "residual": rng.choice(["f32", "bf16", "none"])}
        return case if op == "norm train" else dict(case, group=rng.choice([-1, -1, 0, 128]))
    if op in ("attention", "attention train", "attention step"):
        heads = _log_int(rng, 1, 96)
        parts = [h for h in range(1, heads + 1) if heads % h == 0]
        case = {"op": op, "batch": _log_int(rng, 1, 128 if op == "attention step" else 6), "heads": heads,
                "q_heads": rng.choice([heads, rng.choice(parts)]), "k_heads": rng.choice([heads, rng.choice(parts)]),
                "v_heads": rng.choice([heads, rng.choice(parts)]), "key_dim": 16 * rng.randint(1, 8),
                "value_dim": 16 * rng.randint(1, 8), "dtype": dtype}
        if op == "attention step":
            return case
        most = (24 << 20 if op == "attention" else 8 << 20) // (
            case["batch"] * heads * max(case["key_dim"], case["value_dim"]))
        return dict(case, L=_log_int(rng, 1, max(1, min(32768, most))), lens=rng.random() < 0.5, h0=rng.random() < 0.5)
    vocab = _log_int(rng, 1000, 131072)
    if op == "logprobs":
        return {"op": op, "rows": _log_int(rng, 1, min(4096, (16 << 20) // vocab)), "vocab": vocab, "dtype": dtype,
                "top": rng.choice([0, 1, rng.randint(2, 20)]), "masked": rng.random() < 0.5}
    return {"op": op, "rows": _log_int(rng, 1, min(8192, (96 << 20) // vocab)), "vocab": vocab, "dtype": dtype,
            "masked": rng.random() < 0.5}


# ------------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, s, t = case["op"], dict(case), DTYPES[case["dtype"]]

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    def whole(lo, hi, *shape):  # lo <= value < hi
        return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)

    if op in ("norm", "norm train"):
        R, W = case["rows"], case["width"]
        s["x"], s["weight"] = normal(R, W, dtype=t), uniform(0.5, 1.5, W)
        s["stream"] = None
        if case["residual"] != "none":  # a residual stream is larger than what one block adds to it
            s["stream"] = normal(R, W, dtype=DTYPES[case["residual"]], scale=4.0)
        if op == "norm train":
            s["dout"] = normal(R, W, dtype=t)
            s["dstream"] = normal(R, W, dtype=s["stream"].dtype) if s["stream"] is not None else None
        return s
    if op in ("logprobs", "logprobs train"):
        R, V = case["rows"], case["vocab"]
        s["logits"] = normal(R, V, dtype=t, scale=2.5)
        s["tokens"] = whole(0, V, R)
        if case["masked"]:
            s["logits"][:, whole(0, 4, V) == 0] = -math.inf
            s["logits"].scatter_(1, s["tokens"].long()[:, None], 1.0)  # a given token is one that was allowed
        if op == "logprobs train":
            s["dlogprobs"], s["dentropy"] = normal(R), normal(R, scale=0.01)
        return s
    B, H, K, V = case["batch"], case["heads"], case["key_dim"], case["value_dim"]
    lead = (B,) if op == "attention step" else (B, case["L"])
    s["q"], s["k"] = normal(*lead, case["q_heads"], K, dtype=t), normal(*lead, case["k_heads"], K, dtype=t)
    s["v"] = normal(*lead, case["v_heads"], V, dtype=t)
    # each head's memory, from about 30 steps to 2000
    s["rate"] = -torch.log1p(-torch.exp2(-uniform(5.0, 11.0, H)))
    if op == "attention step":
        s["state"] = normal(B, H, K, V)
        return s
    s["state"] = normal(B, H, K, V) if case["h0"] else None
    s["seq_lens"] = whole(0, case["L"] + 1, B) if case["lens"] else None
    if op == "attention train":
        s["dout"] = normal(B, case["L"], H, V, dtype=t)
        s["dlast"] = normal(B, H, K, V) if case["h0"] else None
    return s


# ------------------------------------------------------------------------------------- passes

def run(s):
    op = s["op"]
    if own:
        return _library(s)
    if op == "norm":
        return _plain_norm(s)
    if op == "norm train":
        return _plain_norm_train(s)
    if op == "attention":
        return _plain_attention(s)
    if op == "attention train":
        return {**_plain_attention(s), **_plain_attention_bwd(s)}
    if op == "attention step":
        return _plain_attention_step(s)
    if op == "logprobs":
        return _plain_logprobs(s)
    return _plain_logprobs_train(s)


def _library(s):
    import selective_state_space_06_amd as mss
    op = s["op"]
    if op == "norm" and s["group"] < 0:
        out, stream = mss.rms_norm_fwd(s["x"], s["weight"], residual=s["stream"], eps=EPS)
        return {"out": out, "residual_out": stream}
    if op == "norm":
        out, scales, stream = mss.rms_norm_fwd_e4m3(s["x"], s["weight"], residual=s["stream"], eps=EPS,
                                                    group=s["group"] or None)
        return {"out": out, "scales": scales, "residual_out": stream}
    if op == "norm train":
        out, stream, rstd = mss.rms_norm_fwd_save(s["x"], s["weight"], residual=s["stream"], eps=EPS)
        g = mss.rms_norm_bwd(s["x"] if stream is None else stream, s["weight"], rstd, s["dout"],
                             dresidual_out=s["dstream"])
        return {"out": out, "residual_out": stream, "dx": g["dx"], "dresidual": g.get("dresidual"),
                "dweight": g["dweight"]}
    if op in ("attention", "attention train"):
        out, last = mss.linear_attention_fwd(s["q"], s["k"], s["v"], s["rate"], initial_state=s["state"],
                                             seq_lens=s["seq_lens"])
        if op == "attention":
            return {"out": out, "last_state": last}
        g = mss.linear_attention_bwd(s["q"], s["k"], s["v"], s["rate"], s["dout"], initial_state=s["state"],
                                     seq_lens=s["seq_lens"], dlast_state=s["dlast"], return_dinitial_state=s["h0"])
        return {"out": out, "last_state": last, "dq": g["dq"], "dk": g["dk"], "dv": g["dv"],
                "dinitial_state": g.get("dinitial_state")}
    if op == "attention step":
        return {"out": mss.linear_attention_update(s["state"], s["q"], s["k"], s["v"], s["rate"]),
                "state": s["state"]}
    if op == "logprobs":
        got = mss.token_logprobs(s["logits"], s["tokens"], top=s["top"])
        return dict(zip(("logprobs", "entropy", "top_logprobs", "top_tokens"), got))
    logprobs, entropy, saved = mss.token_logprobs_save(s["logits"], s["tokens"])
    return {"logprobs": logprobs, "entropy": entropy,
            "dlogits": mss.token_logprobs_bwd(s["logits"], s["tokens"], saved, s["dlogprobs"], s["dentropy"])}


def _stream(s):
    """x, or the residual stream with x added, in the stream's type: what the norm is of."""
    return s["x"] if s["stream"] is None else (s["x"].float() + s["stream"].float()).to(s["stream"].dtype)


def _plain_sum(s):
    z = _stream(s).float()
    return z, torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS)


def _plain_norm(s):
    z, r = _plain_sum(s)
    y = z * r * s["weight"]
    got = {"residual_out": None if s["stream"] is None else z.to(s["stream"].dtype)}
    if s["group"] < 0:
        return {"out": y.to(s["x"].dtype), **got}
    R, W = y.shape
    n = s["group"] or W
    parts = torch.nn.functional.pad(y, (0, -W % n)).reshape(R, -1, n)
    scales = parts.abs().amax(-1).clamp_min(2.0 ** -100) / 448
    q = (parts / scales[..., None]).clamp(-448, 448).reshape(R, -1)[:, :W]
    return {"out": q.contiguous().to(torch.float8_e4m3fn), "scales": scales, **got}


def _plain_norm_train(s):
    z, r = _plain_sum(s)
    zhat, d = z * r, s["dout"].float()
    w = d * s["weight"]
    dz = r * (w - zhat * (w * zhat).mean(-1, keepdim=True))
    got = {"out": (zhat * s["weight"]).to(s["x"].dtype), "residual_out": None, "dresidual": None}
    if s["stream"] is not None:
        dz = dz + s["dstream"].float()
        got["residual_out"], got["dresidual"] = z.to(s["stream"].dtype), dz.to(s["stream"].dtype)
    return {**got, "dx": dz.to(s["x"].dtype), "dweight": (d * zhat).double().sum(0).float()}


def _powers(rate, n):
    """exp(-rate n) per head, in 64 bits and rounded: rate (heads,), n of any shape -> (heads, *n.shape)."""
    return torch.exp(-rate.double().reshape(-1, *[1] * n.dim()) * n.double()).float()


def _plain_decayed(q, k, v, rate, C=128):
    """sum over s <= t of exp(-rate (t - s)) (q_t . k_s) v_s for (batch, heads, L, ...): within chunks by their scores,
    between them by states at the chunks' ends, all chunks at once."""
    B, H, L, _ = q.shape
    pad = -L % C
    q, k, v = (torch.nn.functional.pad(t, (0, 0, 0, pad)).unflatten(2, (-1, C)) for t in (q, k, v))
    n, i = q.shape[2], torch.arange(C, device=q.device)
    near = torch.where(i[:, None] >= i, _powers(rate, (i[:, None] - i).clamp_min(0)), 0.0)
    out = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * near[:, None], v)
    ends = torch.matmul((k * _powers(rate, C - 1 - i)[:, None, :, None]).transpose(-1, -2), v)
    c = torch.arange(n, device=q.device)
    far = torch.where(c[:, None] > c, _powers(rate, C * (c[:, None] - 1 - c).clamp_min(0)), 0.0)
    before = torch.matmul(far, ends.flatten(3)).reshape(ends.shape)
    out = out + torch.matmul(q * _powers(rate, i + 1)[:, None, :, None], before)
    return out.flatten(2, 3)[:, :, :L]


def _plain_heads(s, name):
    """(batch, L, heads, d) -> (batch, every head, L, d) in 32 bits, zeros past the sequences' ends."""
    t = s[name].float().repeat_interleave(s["heads"] // s[name].shape[2], 2).transpose(1, 2)
    return torch.where(_plain_valid(s), t, 0.0)


def _plain_valid(s):
    L = s["q"].shape[1]
    lens = s["seq_lens"] if s["seq_lens"] is not None else torch.full((s["batch"],), L, device="cuda")
    return (torch.arange(L, device="cuda") < lens[:, None])[:, None, :, None]


def _plain_weights(s):
    """exp(-rate n) per (batch, head, step) for the steps up to and with t, and those from t to the end; and for all."""
    L = s["q"].shape[1]
    t = torch.arange(L, device="cuda")
    lens = s["seq_lens"] if s["seq_lens"] is not None else torch.full((s["batch"],), L, device="cuda")
    left = _powers(s["rate"], (lens[:, None] - 1 - t).clamp_min(0)).transpose(0, 1)
    return _powers(s["rate"], t + 1)[None, ..., None], left[..., None], _powers(s["rate"], lens).t()[..., None, None]


def _plain_attention(s):
    q, k, v = (_plain_heads(s, n) for n in ("q", "k", "v"))
    since, left, whole = _plain_weights(s)
    out = _plain_decayed(q, k, v, s["rate"])
    last = torch.matmul((k * left).transpose(-1, -2), v)
    if s["state"] is not None:
        out = out + torch.matmul(q * since, s["state"])
        last = last + whole * s["state"]
    out = out * s["key_dim"] ** -0.5
    return {"out": out.transpose(1, 2).contiguous().to(s["q"].dtype), "last_state": last}


def _plain_attention_bwd(s):
    q, k, v = (_plain_heads(s, n) for n in ("q", "k", "v"))
    d = _plain_heads(s, "dout") * s["key_dim"] ** -0.5
    since, left, whole = _plain_weights(s)
    valid = _plain_valid(s)
    dq = _plain_decayed(d, v, k, s["rate"])
    # backwards in time the same sums: of every step that a key or a value reaches
    dk = _plain_decayed(v.flip(2), d.flip(2), q.flip(2), s["rate"]).flip(2)
    dv = _plain_decayed(k.flip(2), q.flip(2), d.flip(2), s["rate"]).flip(2)
    got = {"dinitial_state": None}
    if s["state"] is not None:
        dq = dq + torch.matmul(d * since, s["state"].transpose(-1, -2))
        dk = dk + torch.matmul(v * left, s["dlast"].transpose(-1, -2))
        dv = dv + torch.matmul(k * left, s["dlast"])
        got["dinitial_state"] = torch.matmul((q * since).transpose(-1, -2), d) + whole * s["dlast"]
    for name, g in (("q", dq), ("k", dk), ("v", dv)):
        g = torch.where(valid, g, 0.0).unflatten(1, (s[name].shape[2], -1)).sum(2)  # over the heads that share it
        got["d" + name] = g.transpose(1, 2).contiguous().to(s[name].dtype)
    return got


def _plain_attention_step(s):
    q, k, v = (s[n].float().repeat_interleave(s["heads"] // s[n].shape[1], 1) for n in ("q", "k", "v"))
    s["state"].mul_(torch.exp(-s["rate"])[:, None, None]).add_(k[..., None] * v[..., None, :])
    out = (s["state"] * q[..., None]).sum(-2) * s["key_dim"] ** -0.5
    return {"out": out.to(s["q"].dtype), "state": s["state"]}


def _plain_softmax(s):
    x = s["logits"].float()
    x = x - x.max(-1, keepdim=True).values
    e = torch.exp(x)
    total = e.sum(-1, keepdim=True)
    lp, p = x - torch.log(total), e / total
    entropy = -torch.where(p > 0, p * lp, 0.0).sum(-1)
    return lp, p, torch.gather(lp, 1, s["tokens"].long()[:, None])[:, 0], entropy


def _plain_logprobs(s):
    lp, _, logprobs, entropy = _plain_softmax(s)
    if not s["top"]:
        return {"logprobs": logprobs, "entropy": entropy}
    # by the logits themselves: equal ones in their own order
    at = torch.sort(s["logits"].float(), dim=-1, descending=True, stable=True).indices[:, :s["top"]]
    top = torch.gather(lp, 1, at)
    return {"logprobs": logprobs, "entropy": entropy, "top_logprobs": top,
            "top_tokens": torch.where(top > -math.inf, at, -1).to(torch.int32)}


def _plain_logprobs_train(s):
    lp, p, logprobs, entropy = _plain_softmax(s)
    d = -p * s["dlogprobs"][:, None]
    d = d.scatter_add(1, s["tokens"].long()[:, None], s["dlogprobs"][:, None])
    d = d - torch.where(p > 0, p * (lp + entropy[:, None]), 0.0) * s["dentropy"][:, None]
    return {"logprobs": logprobs, "entropy": entropy, "dlogits": d.to(s["logits"].dtype)}


# ------------------------------------------------------------------------------ what it takes

def work(case):
    """Each input read once and each output written once; the operations of the formulas (attention's in its
    recurrent form), an exponential, root or division as one."""
    op, e = case["op"], {"f32": 4, "bf16": 2}[case["dtype"]]
    if op in ("norm", "norm train"):
        n, W = case["rows"] * case["width"], case["width"]
        r = {"f32": 4, "bf16": 2, "none": 0}[case["residual"]]
        if op == "norm":
            scales = 4 * case["rows"] * (-(-W // case["group"]) if case["group"] > 0 else 1)
            out = n * e if case["group"] < 0 else n + scales
            return {"bytes": n * (e + 2 * r) + out + 4 * W, "flops": 5 * n}
        # the sum is read again by the backward, as no other tensor holds it
        return {"bytes": n * (4 * e + 4 * r + (r or e)) + 12 * W, "flops": 14 * n}
    if op in ("logprobs", "logprobs train"):
        n = case["rows"] * case["vocab"]
        if op == "logprobs":
            return {"bytes": n * e + case["rows"] * (12 + 8 * case["top"]), "flops": 5 * n}
        return {"bytes": 3 * n * e + 20 * case["rows"], "flops": 12 * n}
    K, V, H, B = case["key_dim"], case["value_dim"], case["heads"], case["batch"]
    n = B * case.get("L", 1)
    ins = n * e * ((case["q_heads"] + case["k_heads"]) * K + case["v_heads"] * V)
    out, state = n * e * H * V, 4 * B * H * K * V
    if op == "attention step":
        return {"bytes": ins + out + 2 * state, "flops": 5 * n * H * K * V}
    if op == "attention":
        return {"bytes": ins + out + state * (2 if case["h0"] else 1), "flops": 4 * n * H * K * V}
    return {"bytes": 2 * ins + 2 * out + state * (4 if case["h0"] else 1), "flops": 14 * n * H * K * V}


# ------------------------------------------------------------------------------------ 64 bits

def _exact_walk(q, k, v, decay, S, ok, first):
    """sum of decayed k v^T seen by q, step by step: q, k, v (batch, heads, L, d); S the state before; a step where `ok`
    is false changes nothing and gives 0.  first: the state enters the first step of a sequence undecayed (the walk
    back from its end).  Returns outputs and the state after."""
    out = q.new_zeros(*q.shape[:3], v.shape[-1])
    began = torch.zeros_like(ok[:, 0]) if first else torch.ones_like(ok[:, 0])
    for t in range(q.shape[2]):
        on = ok[:, t, None, None, None]
        new = torch.where(began[:, None, None, None], decay * S, S) + k[:, :, t, :, None] * v[:, :, t, None, :]
        began = began | ok[:, t]
        S = torch.where(on, new, S)
        out[:, :, t] = torch.where(on, (q[:, :, t, None, :] @ S), 0.0)[:, :, 0]
    return out, S


def _exact_attention(s, case):
    step = case["op"] == "attention step"
    H, K = case["heads"], case["key_dim"]

    def wide(t):
        t = t[:, None] if step else t
        return t.double().movedim(2, 1).repeat_interleave(H // t.shape[2], 1)

    q, k, v = wide(s["q"]), wide(s["k"]), wide(s["v"])
    B, _, L, V = v.shape
    decay = torch.exp(-s["rate"].double())[:, None, None]
    lens = s.get("seq_lens")
    ok = torch.ones(B, L, dtype=torch.bool, device="cuda") if lens is None else \
        torch.arange(L, device="cuda")[None] < lens[:, None]
    S = s["state"].double() if s["state"] is not None else q.new_zeros(B, H, K, V)
    out, last = _exact_walk(q, k, v, decay, S, ok, False)
    out = (out / math.sqrt(K)).movedim(1, 2)
    if step:
        return {"out": out[:, 0], "state": last}
    if case["op"] == "attention":
        return {"out": out, "last_state": last}
    d = wide(s["dout"]) / math.sqrt(K)
    E = s["dlast"].double() if s["dlast"] is not None else torch.zeros_like(S)
    dq, _ = _exact_walk(d, v, k, decay, S.transpose(-1, -2), ok, False)
    back = ok.flip(1)
    dv, G = _exact_walk(k.flip(2), q.flip(2), d.flip(2), decay, E, back, True)
    dk, _ = _exact_walk(v.flip(2), d.flip(2), q.flip(2), decay, E.transpose(-1, -2), back, True)
    some = ok.any(1)[:, None, None, None]

    def shared(g, name):
        n = s[name].shape[2]
        return torch.stack([g[:, h * (H // n):(h + 1) * (H // n)].sum(1) for h in range(n)], 2)

    return {"out": out, "last_state": last, "dq": shared(dq, "q"), "dk": shared(dk.flip(2), "k"),
            "dv": shared(dv.flip(2), "v"),
            "dinitial_state": torch.where(some, decay * G, G) if case["h0"] else None}


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("attention", "attention train", "attention step"):
        return _exact_attention(s, case)
    if op in ("logprobs", "logprobs train"):
        x, at = s["logits"].double(), s["tokens"].long()
        lse = torch.logsumexp(x, -1)
        rows = torch.arange(len(at), device="cuda")
        p = torch.exp(x - lse[:, None])
        logprobs = x[rows, at] - lse
        entropy = lse - torch.where(p > 0, x, 0.0).mul_(p).sum(-1)
        if op == "logprobs":
            got = {"logprobs": logprobs, "entropy": entropy}
            if case["top"]:
                got.update(top_logprobs=x.topk(case["top"], -1).values - lse[:, None], top_tokens=None)
            return got
        # d entropy / dx_v = -p_v (x_v - lse + entropy)
        d = torch.where(p > 0, lse[:, None] - entropy[:, None] - x, 0.0).mul_(s["dentropy"].double()[:, None])
        d = d.sub_(s["dlogprobs"].double()[:, None]).mul_(p)
        d[rows, at] += s["dlogprobs"].double()
        return {"logprobs": logprobs, "entropy": entropy, "dlogits": d}
    z = _stream(s).double()
    W, w = z.shape[1], s["weight"].double()
    r = 1 / torch.sqrt(torch.linalg.vector_norm(z, dim=1, keepdim=True) ** 2 / W + EPS)
    y = z * w * r
    stream = z if s["stream"] is not None else None
    if op == "norm":
        if case["group"] < 0:
            return {"out": y, "residual_out": stream}
        n = case["group"] or W
        scales = torch.stack([c.abs().max(1).values for c in y.split(n, 1)], 1) / 448
        # the quotients before their rounding to 8 bits
        return {"out": y / scales.repeat_interleave(n, 1)[:, :W], "scales": scales, "residual_out": stream}
    d = s["dout"].double()
    # through z r(z): the part along z is taken out
    along = (d * y).sum(1, keepdim=True) * r / W
    dz = r * d * w - along * r * z
    if s["dstream"] is not None:
        dz = dz + s["dstream"].double()
    return {"out": y, "residual_out": stream, "dx": dz, "dresidual": dz if s["stream"] is not None else None,
            "dweight": (d * z * r).sum(0)}
