"""Measured cases of the gated scan, the causal conv's backward and beam search.

Each case is one call (or, for the training cases, a forward with its backward) of an operator on
synthetic data: `run` computes it in its plain form from elementary torch operations (`own` false)
or through the library (`own` true), `exact` from the definition in 64 bits.

gated scan     r = sigmoid(fgate), a = exp(-rate r), h_t = a_t h_{t-1} + sqrt(1 - a_t^2)
               sigmoid(igate_t) x_t, out_t = h_t, per (batch, channel); steps past a sequence's
               length leave the state alone and give 0
conv backward  gradients of y_t = bias + sum_k w_k x_{t-(K-1)+k}, out = silu(y) or y
beam select    the k best continuations of a request's beams by score + log softmax(logits);
               a finished beam has one continuation, its end token at its own score
beam reorder   state[b, j] = state[b, parents[b, j]] for the states of every layer, in place
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # prefill of one layer of the 2.8B shape, a batch of four full prompts
        {"name": "scan layer bf16", "op": "scan", "batch": 4, "d_inner": 5120, "L": 2048, "dtype": "bf16",
         "lens": False, "h0": False},
        # one long document appended to a kept state: few rows, the time axis is the work
        {"name": "scan long f32", "op": "scan", "batch": 1, "d_inner": 1536, "L": 131072, "dtype": "f32",
         "lens": False, "h0": True},
        # a training step of the same layer: forward, then all gradients
        {"name": "train layer bf16", "op": "train", "batch": 4, "d_inner": 5120, "L": 2048, "dtype": "bf16",
         "lens": False, "h0": False},
        # a training step on a batch of different lengths whose rows are no whole vectors
        {"name": "train ragged f32", "op": "train", "batch": 3, "d_inner": 1531, "L": 2041, "dtype": "f32",
         "lens": True, "h0": True},
        # one token for one request: latency
        {"name": "step one f32", "op": "step", "batch": 1, "d_inner": 1536, "dtype": "f32"},
        # one token for a batch of 64 requests of the 2.8B width
        {"name": "step batch bf16", "op": "step", "batch": 64, "d_inner": 5120, "dtype": "bf16"},
        # the conv in front of the layer above, in training
        {"name": "conv layer bf16", "op": "conv", "batch": 4, "d_inner": 5120, "L": 2048, "K": 4, "dtype": "bf16",
         "silu": True, "states": False},
        # the second chunk of a chunked training sequence: carried window in, gradient of it out
        {"name": "conv ragged f32", "op": "conv", "batch": 8, "d_inner": 1536, "L": 2047, "K": 4, "dtype": "f32",
         "silu": True, "states": True},
        # one request, four beams: latency
        {"name": "select one bf16", "op": "select", "batch": 1, "beams": 4, "vocab": 32768, "dtype": "bf16",
         "finished": False},
        # a full batch with eight beams each over a large odd vocabulary, some beams at their end
        {"name": "select batch f32", "op": "select", "batch": 64, "beams": 8, "vocab": 128007, "dtype": "f32",
         "finished": True},
        # four beams of one request through the 24 layers of the 130M shape
        {"name": "reorder one", "op": "reorder", "batch": 1, "beams": 4, "d_inner": 1536, "d_state": 16, "K": 4,
         "layers": 24},
        # sixteen requests of four beams, eight layers of the 2.8B shape
        {"name": "reorder batch", "op": "reorder", "batch": 16, "beams": 4, "d_inner": 5120, "d_state": 16, "K": 4,
         "layers": 8},
    ]


def _log_int(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "train", "step", "conv", "select", "reorder"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("scan", "train", "conv"):
        batch, d_inner = _log_int(rng, 1, 8), _log_int(rng, 64, 5120)
        most = (200 << 20 if op == "scan" else 40 << 20) // (batch * d_inner)
        L = _log_int(rng, 1, min(131072, most))
        case = {"op": op, "batch": batch, "d_inner": d_inner, "L": L, "dtype": dtype}
        if op == "conv":
            return dict(case, K=rng.randint(2, 4), silu=rng.random() < 0.7, states=rng.random() < 0.5)
        return dict(case, lens=rng.random() < 0.5, h0=rng.random() < 0.5)
    if op == "step":
        return {"op": op, "batch": _log_int(rng, 1, 256), "d_inner": _log_int(rng, 64, 5120), "dtype": dtype}
    if op == "select":
        batch, beams = _log_int(rng, 1, 64), _log_int(rng, 2, 16)
        most = (64 << 20) // (batch * beams)
        return {"op": op, "batch": batch, "beams": beams, "vocab": _log_int(rng, 1000, min(131072, most)),
                "dtype": dtype, "finished": rng.random() < 0.5}
    return {"op": op, "batch": _log_int(rng, 1, 16), "beams": _log_int(rng, 2, 8), "d_inner": _log_int(rng, 64, 5120),
            "d_state": rng.choice([16, 32, 64]), "K": rng.randint(2, 4), "layers": rng.randint(1, 8)}


# ------------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], dict(case)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    def whole(lo, hi, *shape):  # lo <= value < hi
        return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)

    if op in ("scan", "train"):
        B, D, L, t = case["batch"], case["d_inner"], case["L"], DTYPES[case["dtype"]]
        s["x"], s["fgate"], s["igate"] = (normal(B, D, L, dtype=t) for _ in range(3))
        # a decay between 0.9 and 0.999 where the gate is fully open: memories of 10 to 1000 steps
        s["rate"] = -torch.log(uniform(0.9, 0.999, D))
        s["state"] = normal(B, D) if case["h0"] else None
        s["seq_lens"] = whole(0, L + 1, B) if case["lens"] else None
        if op == "train":
            s["dout"] = normal(B, D, L, dtype=t)
            s["dlast"] = normal(B, D) if case["h0"] else None
    elif op == "step":
        B, D, t = case["batch"], case["d_inner"], DTYPES[case["dtype"]]
        s["state"] = normal(B, D)
        s["x"], s["fgate"], s["igate"] = (normal(B, D, dtype=t) for _ in range(3))
        s["rate"] = -torch.log(uniform(0.9, 0.999, D))
    elif op == "conv":
        B, D, L, K, t = case["batch"], case["d_inner"], case["L"], case["K"], DTYPES[case["dtype"]]
        s["x"], s["dout"] = normal(B, D, L, dtype=t), normal(B, D, L, dtype=t)
        s["weight"], s["bias"] = normal(D, K, scale=0.5), normal(D, scale=0.1)
        s["state"] = normal(B, D, K - 1, dtype=t) if case["states"] else None
        s["dfinal"] = normal(B, D, K - 1, dtype=t) if case["states"] else None
    elif op == "select":
        B, N, V, t = case["batch"], case["beams"], case["vocab"], DTYPES[case["dtype"]]
        s["logits"] = normal(B, N, V, dtype=t, scale=2.5)
        s["scores"] = -uniform(1.0, 20.0, B, N)
        s["done"] = (whole(0, 4, B, N) == 0).to(torch.int32) if case["finished"] else None
        s["end_token"] = V // 3
    else:
        B, N, D = case["batch"], case["beams"], case["d_inner"]
        s["parents"] = whole(0, N, B, N)
        s["states"] = [normal(B * N, D, case["d_state"]) for _ in range(case["layers"])]
        s["states"] += [normal(B * N, D, case["K"] - 1, dtype=torch.bfloat16) for _ in range(case["layers"])]
    return s


# ------------------------------------------------------------------------------------- passes

def run(s):
    op = s["op"]
    if own:
        import selective_state_space_06_amd as mss
    if op == "scan":
        if own:
            out, last = mss.gated_scan_fwd(s["x"], s["fgate"], s["igate"], s["rate"], initial_state=s["state"],
                                           seq_lens=s["seq_lens"])
        else:
            out, last = _plain_scan(s)
        return {"out": out, "last_state": last}
    if op == "train":
        if own:
            out, last, saved = mss.gated_scan_fwd_save(s["x"], s["fgate"], s["igate"], s["rate"],
                                                       initial_state=s["state"], seq_lens=s["seq_lens"])
            g = mss.gated_scan_bwd(s["x"], s["fgate"], s["igate"], s["rate"], s["dout"], seq_lens=s["seq_lens"],
                                   dlast_state=s["dlast"], return_dinitial_state=s["h0"], saved_states=saved)
        else:
            out, last, g = _plain_train(s)
        return {"out": out, "last_state": last, "dx": g["dx"], "dfgate": g["dfgate"], "digate": g["digate"],
                "drate": g["drate"], "dinitial_state": g.get("dinitial_state")}
    if op == "step":
        if own:
            out = mss.gated_state_update(s["state"], s["x"], s["fgate"], s["igate"], s["rate"])
        else:
            a, v, _ = _plain_gates(s["x"], s["fgate"], s["igate"], s["rate"])
            s["state"].mul_(a).add_(v)
            out = s["state"].to(s["x"].dtype)
        return {"out": out, "state": s["state"]}
    if op == "conv":
        if own:
            g = mss.causal_conv1d_bwd(s["x"], s["weight"], s["dout"], bias=s["bias"], initial_state=s["state"],
                                      silu=s["silu"], dfinal_state=s["dfinal"], return_dinitial_state=s["states"])
        else:
            g = _plain_conv(s)
        return {"dx": g["dx"], "dweight": g["dweight"], "dbias": g["dbias"],
                "dinitial_state": g.get("dinitial_state")}
    if op == "select":
        if own:
            got = mss.beam_select(s["logits"], s["scores"], finished=s["done"],
                                  end_token=s["end_token"] if s["finished"] else None)
        else:
            got = _plain_select(s)
        return dict(zip(("scores", "parents", "tokens", "finished"), got))
    if own:
        mss.beam_reorder(s["states"], s["parents"])
    else:
        B, N = s["parents"].shape
        at = (s["parents"] + torch.arange(B, device="cuda", dtype=torch.int32)[:, None] * N).reshape(-1)
        [t.copy_(t.index_select(0, at)) for t in s["states"]]
    return s["states"]


def _plain_gates(x, fgate, igate, rate):
    """a, the input term, and sigmoid(fgate), in 32 bits; rate broadcast over the last axis of x."""
    r = 1 / (1 + torch.exp(-fgate.float()))
    decay = rate * r
    v = torch.sqrt(-torch.expm1(-2 * decay)) / (1 + torch.exp(-igate.float())) * x.float()
    return torch.exp(-decay), v, r


def _plain_recurrence(a, v):
    """h_t = a_t h_{t-1} + v_t along the last axis, by doubling: after a round every step holds the
    combined transition of twice as many steps."""
    step, L = 1, a.shape[-1]
    while step < L:
        v = torch.cat([v[..., :step], v[..., step:] + a[..., step:] * v[..., :-step]], -1)
        a = torch.cat([a[..., :step], a[..., step:] * a[..., :-step]], -1)
        step *= 2
    return v


def _plain_valid(s):
    L = s["x"].shape[-1]
    if s["seq_lens"] is None:
        return None
    return (torch.arange(L, device="cuda") < s["seq_lens"][:, None])[:, None, :]


def _plain_forward(s):
    a, v, r = _plain_gates(s["x"], s["fgate"], s["igate"], s["rate"][:, None])
    valid = _plain_valid(s)
    if valid is not None:
        a, v = torch.where(valid, a, 1.0), torch.where(valid, v, 0.0)
    if s["state"] is not None:
        v = torch.cat([v[..., :1] + a[..., :1] * s["state"][..., None], v[..., 1:]], -1)
    return a, r, valid, _plain_recurrence(a, v)


def _plain_scan(s):
    a, r, valid, h = _plain_forward(s)
    out = h if valid is None else torch.where(valid, h, 0.0)
    return out.to(s["x"].dtype), h[..., -1].clone()


def _plain_train(s):
    x, t = s["x"].float(), s["x"].dtype
    a, r, valid, h = _plain_forward(s)
    h0 = torch.zeros_like(h[..., :1]) if s["state"] is None else s["state"][..., None]
    before = torch.cat([h0, h[..., :-1]], -1)
    # the adjoint: G_t = dout_t + a_{t+1} G_{t+1}
    d = s["dout"].float()
    if valid is not None:
        d = torch.where(valid, d, 0.0)
    if s["dlast"] is not None:
        d = torch.cat([d[..., :-1], d[..., -1:] + s["dlast"][..., None]], -1)
    later = torch.cat([a[..., 1:], torch.zeros_like(a[..., :1])], -1)
    G = _plain_recurrence(later.flip(-1), d.flip(-1)).flip(-1)
    decay = s["rate"][:, None] * r
    m = torch.sqrt(-torch.expm1(-2 * decay))
    p = 1 / (1 + torch.exp(-s["igate"].float()))
    e = torch.exp(-decay)
    into = torch.where(m > 0, e * e / m, 0.0)  # d sqrt(1 - a^2) / d decay
    ddecay = G * (into * p * x - e * before)
    g = {"dx": G * m * p, "digate": G * m * p * (1 - p) * x, "dfgate": ddecay * decay * (1 - r), "ddecay": ddecay * r}
    if valid is not None:
        g = {k: torch.where(valid, v, 0.0) for k, v in g.items()}
    drate = g.pop("ddecay").double().sum((0, 2)).float()
    g = {k: v.to(t) for k, v in g.items()}
    g["drate"] = drate
    if s["h0"]:
        g["dinitial_state"] = a[..., 0] * G[..., 0]
    out = h if valid is None else torch.where(valid, h, 0.0)
    return out.to(t), h[..., -1].clone(), g


def _plain_conv(s):
    x, d, w, K = s["x"].float(), s["dout"].float(), s["weight"], s["K"]
    B, D, L = x.shape
    before = x.new_zeros(B, D, K - 1) if s["state"] is None else s["state"].float()
    window = torch.cat([before, x], -1)
    if s["silu"]:
        y = s["bias"][:, None] + sum(w[:, k, None] * window[..., k:k + L] for k in range(K))
        p = 1 / (1 + torch.exp(-y))
        d = d * p * (1 + y * (1 - p))
    dwindow = sum(torch.nn.functional.pad(w[:, k, None] * d, (k, K - 1 - k)) for k in range(K))
    if s["dfinal"] is not None:
        dwindow = torch.cat([dwindow[..., :L], dwindow[..., L:] + s["dfinal"].float()], -1)
    g = {"dx": dwindow[..., K - 1:].to(s["x"].dtype),
         "dweight": torch.stack([(d * window[..., k:k + L]).double().sum((0, 2)) for k in range(K)], -1).float(),
         "dbias": d.double().sum((0, 2)).float()}
    if s["states"]:
        g["dinitial_state"] = dwindow[..., :K - 1].to(s["x"].dtype)
    return g


def _plain_select(s):
    # in 64 bits: equal and nearly equal scores decide the order
    x, scores = s["logits"].double(), s["scores"].double()
    B, N, V = x.shape
    top = x.max(-1, keepdim=True).values
    total = scores[..., None] + (x - (top + torch.log(torch.exp(x - top).sum(-1, keepdim=True))))
    if s["done"] is not None:
        end = torch.arange(V, device="cuda") == s["end_token"]
        total = torch.where(s["done"].bool()[..., None], torch.where(end, scores[..., None], -math.inf), total)
    best, at = torch.sort(total.reshape(B, N * V), dim=-1, descending=True, stable=True)
    best, at = best[:, :N], at[:, :N]
    got = (best.float(), (at // V).to(torch.int32), (at % V).to(torch.int32))
    if s["done"] is None:
        return got
    ended = (torch.gather(s["done"], 1, at // V) != 0) | (at % V == s["end_token"])
    return got + (ended.to(torch.int32),)


# ------------------------------------------------------------------------------ what it takes

def work(case):
    """Each input read once and each output written once; the operations of the formulas, an
    exponential, root or division as one."""
    op, e = case["op"], {"f32": 4, "bf16": 2}.get(case.get("dtype"), 4)
    if op in ("scan", "train"):
        B, D, n = case["batch"], case["d_inner"], case["batch"] * case["d_inner"] * case["L"]
        rows = B * D * 4
        if op == "scan":
            return {"bytes": 4 * n * e + rows * (2 if case["h0"] else 1) + 4 * D, "flops": 16 * n}
        return {"bytes": 8 * n * e + rows * (4 if case["h0"] else 1) + 8 * D, "flops": 50 * n}
    if op == "step":
        n = case["batch"] * case["d_inner"]
        return {"bytes": n * (8 + 4 * e) + 4 * case["d_inner"], "flops": 16 * n}
    if op == "conv":
        n, K = case["batch"] * case["d_inner"] * case["L"], case["K"]
        states = 3 * case["batch"] * case["d_inner"] * (K - 1) * e if case["states"] else 0
        return {"bytes": 3 * n * e + states + 8 * case["d_inner"] * (K + 1), "flops": n * (6 * K + 8)}
    if op == "select":
        n = case["batch"] * case["beams"] * case["vocab"]
        return {"bytes": n * e + case["batch"] * case["beams"] * 20, "flops": 4 * n}
    # a beam that keeps its own state need not be touched: one in `beams`
    per = case["batch"] * case["beams"] * case["d_inner"] * (4 * case["d_state"] + 2 * (case["K"] - 1))
    return {"bytes": 2 * case["layers"] * per * (1 - 1 / case["beams"]), "flops": 0}


# ------------------------------------------------------------------------------------ 64 bits

def _exact_recurrence(a, v, h0):
    """h_t = a_t h_{t-1} + v_t step by step in two levels: all blocks of the time axis at once from
    a zero state, then the blocks in order, each from the end of the one before."""
    rows, L = a.shape
    T = max(1, int(math.isqrt(L)))
    C = -(-L // T)
    a = torch.cat([a, a.new_ones(rows, C * T - L)], 1).reshape(rows, C, T)
    v = torch.cat([v, v.new_zeros(rows, C * T - L)], 1).reshape(rows, C, T)
    h, p = torch.empty_like(v), torch.empty_like(a)
    state, product = torch.zeros_like(v[..., 0]), torch.ones_like(v[..., 0])
    for t in range(T):
        state = a[..., t] * state + v[..., t]
        product = product * a[..., t]
        h[..., t], p[..., t] = state, product
    carry = h0
    for c in range(C):
        h[:, c] += p[:, c] * carry[:, None]
        carry = h[:, c, -1]
    return h.reshape(rows, C * T)[:, :L]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("scan", "train", "step"):
        shape = s["x"].shape
        B, D = shape[:2]
        L = 1 if op == "step" else shape[2]
        x, f, i = (s[k].double().reshape(B * D, L) for k in ("x", "fgate", "igate"))
        rate = s["rate"].double().repeat(B)[:, None]
        r, p = torch.special.expit(f), torch.special.expit(i)
        a = torch.exp(-rate * r)
        m = torch.sqrt(-torch.special.expm1(-2 * rate * r))
        lens = s.get("seq_lens")
        lens = torch.full((B,), L, device="cuda") if lens is None else lens
        ok = torch.arange(L, device="cuda")[None] < lens.repeat_interleave(D)[:, None]
        a1, v = torch.where(ok, a, 1.0), torch.where(ok, m * p * x, 0.0)
        h0 = s["state"].double().reshape(-1) if s["state"] is not None else x.new_zeros(B * D)
        h = _exact_recurrence(a1, v, h0)
        last = h[:, -1].reshape(B, D)
        out = torch.where(ok, h, 0.0).reshape(shape)
        if op == "step":
            return {"out": out, "state": last}
        if op == "scan":
            return {"out": out, "last_state": last}
        d = torch.where(ok, s["dout"].double().reshape(B * D, L), 0.0)
        dlast = s["dlast"].double().reshape(-1) if s["dlast"] is not None else x.new_zeros(B * D)
        # reversed in time the adjoint of the step's input, w_t = a_t G_t, is a recurrence of its own:
        # G_t = d_t + w_{t+1}, with the gradient of the last state as what follows the last step
        w = _exact_recurrence(a1.flip(1), (a1 * d).flip(1), dlast).flip(1)
        G = d + torch.cat([w[:, 1:], dlast[:, None]], 1)
        before = torch.cat([h0[:, None], h[:, :-1]], 1)
        dm = G * p * x
        ds = torch.where(ok, dm * a * a / m - G * a * before, 0.0)
        dx, di = torch.where(ok, G * m * p, 0.0), torch.where(ok, G * m * x * p * (1 - p), 0.0)
        return {"out": out, "last_state": last, "dx": dx.reshape(shape), "digate": di.reshape(shape),
                "dfgate": (ds * rate * r * (1 - r)).reshape(shape),
                "drate": (ds * r).reshape(B, D, L).sum((0, 2)),
                "dinitial_state": w[:, 0].reshape(B, D) if case["h0"] else None}
    if op == "conv":
        B, D, L = s["x"].shape
        K, w = case["K"], s["weight"].double()
        head = s["x"].new_zeros(B, D, K - 1) if s["state"] is None else s["state"]
        taps = torch.cat([head, s["x"]], -1).double().unfold(-1, K, 1)  # (B, D, L, K)
        d = s["dout"].double()
        if case["silu"]:
            y = (taps * w[:, None, :]).sum(-1) + s["bias"].double()[:, None]
            q = torch.special.expit(y)
            d = d * (q + y * q * torch.special.expit(-y))
        # input j of the window row feeds steps j - (K-1) .. j: the same taps, reversed, over d
        around = torch.nn.functional.pad(d, (K - 1, K - 1)).unfold(-1, K, 1)
        dwindow = (around * w.flip(1)[:, None, :]).sum(-1)
        if s["dfinal"] is not None:
            dwindow[..., L:] += s["dfinal"].double()
        return {"dx": dwindow[..., K - 1:], "dweight": (taps * d[..., None]).sum((0, 2)), "dbias": d.sum((0, 2)),
                "dinitial_state": dwindow[..., :K - 1] if case["states"] else None}
    if op == "select":
        x, base = s["logits"].double(), s["scores"].double()
        N = x.shape[1]
        best = base[..., None] + x.topk(N, -1).values - torch.logsumexp(x, -1, keepdim=True)
        if s["done"] is not None:
            only = torch.full_like(best, -math.inf)
            only[..., 0] = base
            best = torch.where(s["done"].bool()[..., None], only, best)
        best = best.flatten(1).topk(N, -1).values
        return {"scores": best, "parents": None, "tokens": None, "finished": None}
    B, N = s["parents"].shape
    at = s["parents"].long()
    return [torch.stack([t.double().unflatten(0, (B, N))[b, at[b]] for b in range(B)]).flatten(0, 1)
            for t in s["states"]]
