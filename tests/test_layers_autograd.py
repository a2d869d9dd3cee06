"""What the autograd wrappers of the RMS norm, linear attention and token log probabilities ask of the library when some
outputs are not used and some inputs need no gradients.  No GPU: the launches are recorded and not made."""
import os

import pytest

import selective_state_space_06_amd as mss
from selective_state_space_06_amd import _layers


@pytest.fixture
def calls(monkeypatch):
    if not os.path.exists(mss.LIB_PATH):
        from selective_state_space_06_amd import build
        build.build()
    got = {}
    monkeypatch.setattr(_layers, "_launch", lambda name, x, *args: got.__setitem__(name, args))
    return got


def some(*shape, grad=True):
    import torch
    return torch.ones(shape, requires_grad=grad)


def test_an_unused_stream_has_no_gradient_to_read(calls):
    x, w, r = some(3, 8), some(8), some(3, 8)
    out, stream = mss.RMSNormFunction.apply(x, w, r)
    out.sum().backward()
    z, weight, rstd, dout, dstream, dx, dresidual, dweight, scratch = calls["rms_norm_bwd"]
    assert dstream is None and dweight is not None
    assert x.grad is not None and r.grad is not None and w.grad is not None


def test_a_stream_alone_is_used(calls):
    x, w, r = some(3, 8), some(8), some(3, 8)
    out, stream = mss.RMSNormFunction.apply(x, w, r)
    stream.sum().backward()
    dout, dstream = calls["rms_norm_bwd"][3:5]
    assert not dout.any() and bool((dstream == 1).all())
    assert x.grad is not None and r.grad is not None


def test_a_weight_without_gradient_has_none_made(calls):
    x, w = some(3, 8), some(8, grad=False)
    mss.RMSNormFunction.apply(x, w)[0].sum().backward()
    args = calls["rms_norm_bwd"]
    assert args[7] is None and args[8] is None and w.grad is None  # dweight and its scratch


def test_an_unused_last_state_has_no_gradient_to_read(calls):
    q, k, v, s = some(1, 4, 2, 16), some(1, 4, 2, 16), some(1, 4, 2, 16), some(1, 2, 16, 16)
    rate = some(2, grad=False)
    mss.LinearAttentionFunction.apply(q, k, v, rate, 0.5, s)[0].sum().backward()
    args = calls["linear_attention_bwd"]
    dlast, dinitial = args[8], args[12]
    assert dlast is None and dinitial is not None and s.grad is not None
    mss.LinearAttentionFunction.apply(q, k, v, rate, 0.5, s.detach())[0].sum().backward()
    assert calls["linear_attention_bwd"][12] is None  # a start state that needs no gradient


def test_a_last_state_alone_is_used(calls):
    q, k, v = some(1, 4, 2, 16), some(1, 4, 2, 16), some(1, 4, 2, 16)
    mss.LinearAttentionFunction.apply(q, k, v, some(2, grad=False))[1].sum().backward()
    args = calls["linear_attention_bwd"]
    assert args[7].shape == (1, 4, 2, 16) and not args[7].any() and bool((args[8] == 1).all())


def test_an_unused_entropy_has_no_gradient_to_read(calls):
    import torch
    x, t = some(3, 8), torch.zeros(3, dtype=torch.int32)
    mss.TokenLogprobsFunction.apply(x, t)[0].sum().backward()
    assert calls["token_logprobs_bwd"][4] is None
    mss.TokenLogprobsFunction.apply(x, t)[1].sum().backward()
    dlogprobs, dentropy = calls["token_logprobs_bwd"][3:5]
    assert not dlogprobs.any() and bool((dentropy == 1).all())
