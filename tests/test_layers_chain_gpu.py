"""The RMS norm, linear attention and token log probabilities together, as a language model uses them: a training step's
gradients against the same model in float64, and prefill followed by decoding against the whole sequence at once.

The model in fp32: embedding, two blocks (norm with the residual's addition, projections, attention, projection), norm, head,
log probabilities.  The kernels' own errors are a few 1e-6 of their magnitudes (their tests); torch's fp32 products add about
sqrt(width) 2^-24, and a block's norm divides both by rms values near 1.  Five such stages of 1e-5 each: 1e-4 of the
largest value is the limit, a tenth of what one bf16 rounding would do."""
import math

import pytest

pytestmark = pytest.mark.gpu

B, L, W, H, D, VOCAB = 2, 75, 64, 4, 16, 501


@pytest.fixture(scope="module")
def mss():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_06_amd as m
    m.load_library()
    return m


def weights(dtype, seed=3):
    import torch
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, dtype=torch.float64).to(dtype).cuda()  # noqa: E731
    p = {"embed": n(VOCAB, W), "norm": 1 + 0.1 * n(W), "head": n(W, VOCAB) / math.sqrt(W)}
    for i in range(2):
        p.update({f"norm{i}": 1 + 0.1 * n(W), f"qkv{i}": n(W, 3 * H * D) / math.sqrt(W), f"out{i}": n(H * D, W) / math.sqrt(W)})
    return {k: v.detach().requires_grad_() for k, v in p.items()}


def rates():
    import torch
    return -torch.log1p(-torch.exp2(-torch.arange(3.0, 3.0 + H))).cuda()


def tokens():
    import torch
    return torch.randint(0, VOCAB, (B, L + 1), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()


def model64(p, ids):
    """The same in float64 and elementary operations."""
    import torch

    def norm(z, w):
        return z / torch.sqrt((z * z).mean(-1, keepdim=True) + 1e-5) * w

    i = torch.arange(L, device="cuda")
    near = torch.where(i[:, None] >= i, torch.exp(-rates().double()[:, None, None] * (i[:, None] - i)), 0.0)
    stream = p["embed"][ids[:, :-1].long()]
    for n in range(2):
        qkv = (norm(stream, p[f"norm{n}"]) @ p[f"qkv{n}"]).view(B, L, 3, H, D).permute(2, 0, 3, 1, 4)
        y = ((qkv[0] @ qkv[1].transpose(-1, -2).contiguous()) * near) @ qkv[2] / math.sqrt(D)
        stream = stream + y.transpose(1, 2).reshape(B, L, H * D) @ p[f"out{n}"]
    lp = torch.log_softmax(norm(stream, p["norm"]) @ p["head"], -1)
    return torch.gather(lp, 2, ids[:, 1:].long()[..., None])[..., 0], -(lp.exp() * lp).sum(-1)


def test_training_step(mss):
    import torch
    ids = tokens()
    p, rate = weights(torch.float32), rates()
    x, stream = None, p["embed"][ids[:, :-1].long()]
    for n in range(2):
        if x is None:
            y, _ = mss.RMSNormFunction.apply(stream, p[f"norm{n}"])
        else:
            y, stream = mss.RMSNormFunction.apply(x, p[f"norm{n}"], stream)
        q, k, v = ((y @ p[f"qkv{n}"]).view(B, L, 3, H, D).unbind(2))
        a, _ = mss.LinearAttentionFunction.apply(q.contiguous(), k.contiguous(), v.contiguous(), rate)
        x = a.reshape(B, L, H * D) @ p[f"out{n}"]
    y, _ = mss.RMSNormFunction.apply(x, p["norm"], stream)
    lp, entropy = mss.TokenLogprobsFunction.apply(y @ p["head"], ids[:, 1:].contiguous())
    (-lp.mean() + 0.1 * entropy.mean()).backward()
    r = weights(torch.float64)
    with torch.no_grad():
        [r[k].copy_(v) for k, v in p.items()]
    lp64, en64 = model64(r, ids)
    (-lp64.mean() + 0.1 * en64.mean()).backward()
    assert float((lp - lp64).abs().max()) <= 1e-4 * float(lp64.abs().max())
    for k in p:
        d, top = float((p[k].grad - r[k].grad).abs().max()), float(r[k].grad.abs().max())
        assert top > 0 and d <= 1e-4 * top, (k, d, top)


def test_prefill_then_decode(mss):
    """Bound steps, captured in a graph and replayed a token at a time, go on where the prompt's states end."""
    import torch
    ids, split = tokens(), 40
    p, rate = {k: v.detach() for k, v in weights(torch.float32).items()}, rates()
    lp64, _ = model64({k: v.double() for k, v in p.items()}, ids)
    x, stream, states = None, p["embed"][ids[:, :split].long()], []
    for n in range(2):
        y, s = mss.rms_norm_fwd(stream if x is None else x, p[f"norm{n}"], residual=None if x is None else stream)
        stream = stream if s is None else s
        q, k, v = (t.contiguous() for t in (y @ p[f"qkv{n}"]).view(B, split, 3, H, D).unbind(2))
        a, last = mss.linear_attention_fwd(q, k, v, rate)
        states.append(last)
        x = a.reshape(B, split, H * D) @ p[f"out{n}"]
    y, _ = mss.rms_norm_fwd(x, p["norm"], residual=stream)
    lp, _ = mss.token_logprobs(y @ p["head"], ids[:, 1:split + 1].contiguous())
    lim = 1e-4 * float(lp64.abs().max())
    assert float((lp - lp64[:, :split]).abs().max()) <= lim

    token, target = torch.zeros(B, dtype=torch.int64, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    start = [s.clone() for s in states]

    def step():
        stream, x = p["embed"][token], None
        for n in range(2):
            y, s = mss.rms_norm_fwd(stream if x is None else x, p[f"norm{n}"], residual=None if x is None else stream)
            stream = stream if s is None else s
            q, k, v = (t.contiguous() for t in (y @ p[f"qkv{n}"]).view(B, 3, H, D).unbind(1))
            x = mss.linear_attention_update(states[n], q, k, v, rate).view(B, H * D) @ p[f"out{n}"]
        y, _ = mss.rms_norm_fwd(x, p["norm"], residual=stream)
        return mss.token_logprobs(y @ p["head"], target, top=3)

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # torch's products take their workspaces
    side.synchronize()
    with torch.cuda.graph(graph, stream=side):
        lp, _, top, best = step()
    torch.cuda.synchronize()
    [s.copy_(t) for s, t in zip(states, start)]
    for i in range(split, L):
        token.copy_(ids[:, i])
        target.copy_(ids[:, i + 1])
        graph.replay()
        torch.cuda.synchronize()
        assert float((lp - lp64[:, i]).abs().max()) <= lim, i
        assert bool((top[:, 0] >= lp).all()) and bool((best >= 0).all())


def test_a_written_state_is_refused_by_a_later_backward(mss):
    import torch
    q = torch.randn(1, 8, 2, 16, device="cuda", requires_grad=True)
    k, v, s = torch.randn(1, 8, 2, 16, device="cuda"), torch.randn(1, 8, 2, 16, device="cuda"), torch.zeros(1, 2, 16, 16, device="cuda")
    out, _ = mss.LinearAttentionFunction.apply(q, k, v, torch.full((2,), 0.1, device="cuda"), None, s)
    mss.linear_attention_update(s, *(t[:, 0].contiguous() for t in (k, k, v)), torch.full((2,), 0.1, device="cuda"))
    with pytest.raises(RuntimeError, match="modified"):
        out.sum().backward()
    x = torch.randn(3, 40, device="cuda", requires_grad=True)
    tok = torch.zeros(3, dtype=torch.int32, device="cuda")
    y = x * 1.0
    lp, _ = mss.TokenLogprobsFunction.apply(y, tok)
    with torch.no_grad():
        mss.token_logprobs_bwd(y, tok, mss.token_logprobs_save(y, tok)[2], torch.ones(3, device="cuda"), dlogits=y)
    with pytest.raises(RuntimeError, match="modified"):
        lp.sum().backward()
