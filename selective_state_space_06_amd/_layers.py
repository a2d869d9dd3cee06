"""Torch front end of the RMS norm, linear attention with a decay per head, and token log probabilities (argument
marshalling only, with the rules of _recurrent.py: scratch from torch's allocator on the current stream).
"""
from __future__ import annotations

import ctypes

from ._binding import MssError, _bound_stream, _desc, _note_written, _ref, _refuse_written, load_library
from ._recurrent import _empty_on, _function, _launch, _native, _raise, _same_device, _scratch

NORM_GROUP = 128  # columns that share a scale in grouped 8-bit outputs


# ------------------------------------------------------------------- raw calls (descriptors or None)

def rms_norm_bwd_scratch(rows, width):
    """Floats of scratch mss_rms_norm_bwd needs for dweight."""
    st, n = _native().rms_norm_bwd_scratch(rows, width)
    _raise(st, "mss_rms_norm_bwd_scratch")
    return n


def linear_attention_scratch(batch, L, heads, q_heads, k_heads, v_heads, key_dim, value_dim):
    """(floats of scratch mss_linear_attention_fwd needs, floats mss_linear_attention_bwd needs)."""
    st, fwd, bwd = _native().linear_attention_scratch(batch, L, heads, q_heads, k_heads, v_heads, key_dim, value_dim)
    _raise(st, "mss_linear_attention_scratch")
    return fwd, bwd


def token_logprobs_scratch(rows, vocab, top):
    """Floats of scratch mss_token_logprobs_fwd needs."""
    st, n = _native().token_logprobs_scratch(rows, vocab, top)
    _raise(st, "mss_token_logprobs_scratch")
    return n


def rms_norm_fwd_raw(x, residual, weight, eps, out, residual_out, rstd, scales, stream) -> int:
    return load_library().mss_rms_norm_fwd(_ref(x), _ref(residual), _ref(weight), eps, _ref(out), _ref(residual_out),
                                           _ref(rstd), _ref(scales), stream)


def rms_norm_bwd_raw(z, weight, rstd, dout, dresidual_out, dx, dresidual, dweight, scratch, stream) -> int:
    return load_library().mss_rms_norm_bwd(_ref(z), _ref(weight), _ref(rstd), _ref(dout), _ref(dresidual_out), _ref(dx),
                                           _ref(dresidual), _ref(dweight), _ref(scratch), stream)


def linear_attention_fwd_raw(q, k, v, rate, scale, initial_state, seq_lens, out, last_state, scratch, stream) -> int:
    return load_library().mss_linear_attention_fwd(_ref(q), _ref(k), _ref(v), _ref(rate), scale, _ref(initial_state),
                                                   _ref(seq_lens), _ref(out), _ref(last_state), _ref(scratch), stream)


def linear_attention_bwd_raw(q, k, v, rate, scale, initial_state, seq_lens, dout, dlast_state, dq, dk, dv,
                             dinitial_state, scratch, stream) -> int:
    return load_library().mss_linear_attention_bwd(_ref(q), _ref(k), _ref(v), _ref(rate), scale, _ref(initial_state),
                                                   _ref(seq_lens), _ref(dout), _ref(dlast_state), _ref(dq), _ref(dk),
                                                   _ref(dv), _ref(dinitial_state), _ref(scratch), stream)


def linear_attention_update_raw(state, q, k, v, rate, scale, out, stream) -> int:
    return load_library().mss_linear_attention_update(_ref(state), _ref(q), _ref(k), _ref(v), _ref(rate), scale,
                                                      _ref(out), stream)


def token_logprobs_fwd_raw(logits, tokens, logprobs, entropy, top_logprobs, top_tokens, saved, scratch, stream) -> int:
    return load_library().mss_token_logprobs_fwd(_ref(logits), _ref(tokens), _ref(logprobs), _ref(entropy),
                                                 _ref(top_logprobs), _ref(top_tokens), _ref(saved), _ref(scratch),
                                                 stream)


def token_logprobs_bwd_raw(logits, tokens, saved, dlogprobs, dentropy, dlogits, stream) -> int:
    return load_library().mss_token_logprobs_bwd(_ref(logits), _ref(tokens), _ref(saved), _ref(dlogprobs),
                                                 _ref(dentropy), _ref(dlogits), stream)


# --------------------------------------------------------------------------------------- RMS norm

def _given(*outputs):
    """Those of a caller's outputs that there are, checked."""
    given = [t for t in outputs if t is not None]
    _refuse_written(*given)
    return given


def _norm_fwd(x, weight, residual, eps, out, residual_out, rstd, scales):
    _launch("rms_norm_fwd", x, x, residual, weight, eps, out, residual_out, rstd, scales)


def _stream_out(residual, residual_out):
    import torch
    if residual is None or residual_out is not None:
        return residual_out
    return torch.empty_like(residual, memory_format=torch.contiguous_format)


def rms_norm_fwd(x, weight, residual=None, eps=1e-5, out=None, residual_out=None):
    """RMS norm (mss_rms_norm_fwd) on the current stream of x's device: z = x + residual in residual's type (x without
    residual), out = z / sqrt(mean z^2 + eps) weight over the last dimension.

    x: (..., width) float32 or bfloat16, 2 to 4 dimensions; weight: (width,) float32; residual: x's shape, float32 or
    bfloat16.  Returns (out, residual_out): out in x's dtype, residual_out the new residual stream in residual's (None
    without residual).  residual_out=residual updates the stream in place."""
    import torch
    given = () if out is residual_out is None else _given(out, residual_out)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    residual_out = _stream_out(residual, residual_out)
    _norm_fwd(x, weight, residual, eps, out, residual_out, None, None)
    if given:
        _note_written(given)
    return out, residual_out


def rms_norm_fwd_e4m3(x, weight, residual=None, eps=1e-5, group=None, out=None, scales=None, residual_out=None):
    """rms_norm_fwd with its output in 8 bits: returns (out, scales, residual_out), out torch.float8_e4m3fn and
    scales float32 such that out * scales is the norm: scales (..., 1), one a row, or with group=128
    (..., ceil(width / 128)), one for each 128 columns."""
    import torch
    if group not in (None, NORM_GROUP):
        raise ValueError(f"a scale is for a row (group=None) or for {NORM_GROUP} columns, got group={group}")
    given = () if out is scales is residual_out is None else _given(out, scales, residual_out)
    if out is None:
        out = torch.empty_like(x, dtype=torch.float8_e4m3fn, memory_format=torch.contiguous_format)
    if scales is None:
        parts = 1 if group is None else -(-x.shape[-1] // NORM_GROUP)
        scales = x.new_empty((*x.shape[:-1], parts), dtype=torch.float32)
    residual_out = _stream_out(residual, residual_out)
    _norm_fwd(x, weight, residual, eps, out, residual_out, None, scales)
    if given:
        _note_written(given)
    return out, scales, residual_out


def rms_norm_fwd_save(x, weight, residual=None, eps=1e-5, out=None, residual_out=None, rstd=None):
    """rms_norm_fwd that also writes what its backward needs: returns (out, residual_out, rstd), rstd (...) float32."""
    import torch
    given = () if out is residual_out is rstd is None else _given(out, residual_out, rstd)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    if rstd is None:
        rstd = x.new_empty(x.shape[:-1], dtype=torch.float32)
    residual_out = _stream_out(residual, residual_out)
    _norm_fwd(x, weight, residual, eps, out, residual_out, rstd, None)
    if given:
        _note_written(given)
    return out, residual_out, rstd


def rms_norm_bwd(z, weight, rstd, dout, dresidual_out=None, return_dresidual=None, return_dweight=True):
    """Gradients of rms_norm_fwd for L = sum(dout * out) + sum(dresidual_out * residual_out), on the current stream.
    z: the forward's residual_out, or its x without residual; rstd: as rms_norm_fwd_save wrote it.  Returns a dict: dx
    in dout's dtype, dweight (width,) float32 (unless return_dweight is false) and, with return_dresidual (None: when
    dresidual_out is given), dresidual in z's dtype (the same tensor as dx where that is dout's)."""
    import torch
    if return_dresidual is None:
        return_dresidual = dresidual_out is not None
    g = dict(dx=torch.empty_like(dout, memory_format=torch.contiguous_format))
    if return_dweight:
        g["dweight"] = torch.empty_like(weight, memory_format=torch.contiguous_format)
    own = None
    if return_dresidual:
        if z.dtype != dout.dtype:
            own = torch.empty_like(z, memory_format=torch.contiguous_format)
        g["dresidual"] = g["dx"] if own is None else own
    # sizes that the query refuses are refused by the call itself, with its own status
    width = z.shape[-1] if z.ndim else 0
    floats = rms_norm_bwd_scratch(z.numel() // width, width) if return_dweight and 1 <= width <= 16384 else 0
    _launch("rms_norm_bwd", z, z, weight, rstd, dout, dresidual_out, g["dx"], own, g.get("dweight"),
            _scratch(floats, z.device))
    return g


# ------------------------------------------------------------------------------- linear attention

def _attention_floats(q, k, v, rate):
    """Floats of scratch of the forward and of the backward; none for what the call itself refuses, with its own status."""
    if q.ndim == 4 and k.ndim == 4 and v.ndim == 4 and rate.ndim == 1:
        batch, L, q_heads, key_dim = q.shape
        _, _, v_heads, value_dim = v.shape
        st, fwd, bwd = _native().linear_attention_scratch(batch, L, rate.shape[0], q_heads, k.shape[2], v_heads, key_dim,
                                                          value_dim)
        if st == 0:
            return fwd, bwd
    return 0, 0


def _scale_of(scale, q):
    return q.shape[-1] ** -0.5 if scale is None and q.ndim and q.shape[-1] else 1.0 if scale is None else float(scale)


def linear_attention_fwd(q, k, v, rate, scale=None, initial_state=None, seq_lens=None, return_last_state=True, out=None,
                         last_state=None):
    """Linear attention with one decay per head (mss_linear_attention_fwd) on the current stream of q's device:
    S_t = exp(-rate) S_{t-1} + k_t v_t^T, out_t = scale S_t^T q_t (scale: key_dim^-0.5 by default).

    q: (batch, L, q_heads, key_dim), k: (batch, L, k_heads, key_dim), v: (batch, L, v_heads, value_dim), float32 or
    bfloat16; rate: (heads,) float32, not negative; every number of heads divides heads, and neighbours share.
    key_dim and value_dim are multiples of 16 up to 128.  initial_state: (batch, heads, key_dim, value_dim) float32
    (None: zeros); seq_lens: (batch,) int32 on the device (None: all L; outputs past a sequence's end are 0).  Returns
    out (batch, L, heads, value_dim) in q's dtype, or (out, last_state) with last_state shaped like initial_state."""
    import torch
    given = () if out is last_state is None else _given(out, last_state)
    if out is None:
        out = q.new_empty((*q.shape[:2], rate.shape[0], v.shape[-1]))
    if return_last_state and last_state is None:
        last_state = q.new_empty((q.shape[0], rate.shape[0], q.shape[-1], v.shape[-1]), dtype=torch.float32)
    floats, _ = _attention_floats(q, k, v, rate)
    _launch("linear_attention_fwd", q, q, k, v, rate, _scale_of(scale, q), initial_state, seq_lens, out,
            last_state if return_last_state else None, _scratch(floats, q.device))
    if given:
        _note_written(given)
    return (out, last_state) if return_last_state else out


def linear_attention_bwd(q, k, v, rate, dout, scale=None, initial_state=None, seq_lens=None, dlast_state=None,
                         return_dinitial_state=False):
    """Gradients of linear_attention_fwd for L = sum(dout * out) + sum(dlast_state * last_state), on the current stream.
    Returns a dict: dq, dk, dv in q's dtype (a shared head has the sum over those that share it) and, with
    return_dinitial_state, dinitial_state (batch, heads, key_dim, value_dim) float32.  The decay has no gradient."""
    import torch
    g = {"d" + n: torch.empty_like(t, memory_format=torch.contiguous_format) for n, t in (("q", q), ("k", k), ("v", v))}
    if return_dinitial_state:
        g["dinitial_state"] = q.new_empty((q.shape[0], rate.shape[0], q.shape[-1], v.shape[-1]), dtype=torch.float32)
    _, floats = _attention_floats(q, k, v, rate)
    _launch("linear_attention_bwd", q, q, k, v, rate, _scale_of(scale, q), initial_state, seq_lens, dout, dlast_state,
            g["dq"], g["dk"], g["dv"], g.get("dinitial_state"), _scratch(floats, q.device))
    return g


def linear_attention_update(state, q, k, v, rate, scale=None, out=None):
    """One token of linear attention (mss_linear_attention_update) on the current stream; `state`
    (batch, heads, key_dim, value_dim) float32 is updated in place.  q: (batch, q_heads, key_dim), k: (batch, k_heads,
    key_dim), v: (batch, v_heads, value_dim).  Returns out (batch, heads, value_dim) in q's dtype."""
    written = (state,) if out is None else (state, out)
    _refuse_written(*written)
    if out is None:
        out = q.new_empty((q.shape[0], rate.shape[0], v.shape[-1]))
    _launch("linear_attention_update", q, state, q, k, v, rate, _scale_of(scale, q), out)
    _note_written(written)
    return out


# -------------------------------------------------------------------------- token log probabilities

def _logprobs_fwd(logits, tokens, top, logprobs, entropy, top_logprobs, top_tokens, saved):
    ok = logits.ndim >= 2 and logits.shape[-1] >= 1 and 0 <= top <= 64
    floats = token_logprobs_scratch(logits.numel() // logits.shape[-1], logits.shape[-1], top) if ok else 0
    _launch("token_logprobs_fwd", logits, logits, tokens, logprobs, entropy, top_logprobs, top_tokens, saved,
            _scratch(floats, logits.device))


def _per_token(tokens):
    import torch
    first = torch.empty_like(tokens, dtype=torch.float32, memory_format=torch.contiguous_format)
    return first, torch.empty_like(first)


def token_logprobs(logits, tokens, top=0):
    """Log probabilities of given tokens (mss_token_logprobs_fwd), on the current stream: returns (logprobs, entropy),
    or with top > 0 (at most 64) (logprobs, entropy, top_logprobs, top_tokens).

    logits: (..., vocab) float32 or bfloat16, 2 to 4 dimensions; tokens: (...) int32 (one outside [0, vocab) has log
    probability 0).  logprobs, entropy: (...) float32; top_logprobs (..., top) float32 and top_tokens (..., top) int32:
    each row's most probable tokens, best first, equal ones by token; -inf and -1 where there are no more."""
    import torch
    logprobs, entropy = _per_token(tokens)
    tops = None, None
    if top:
        shape = (*tokens.shape, top)
        tops = tokens.new_empty(shape, dtype=torch.float32), tokens.new_empty(shape, dtype=torch.int32)
    _logprobs_fwd(logits, tokens, int(top), logprobs, entropy, *tops, None)
    return (logprobs, entropy, *tops) if top else (logprobs, entropy)


def token_logprobs_save(logits, tokens):
    """token_logprobs that also returns what its backward needs: (logprobs, entropy, saved), saved (..., 3) float32."""
    import torch
    logprobs, entropy = _per_token(tokens)
    saved = tokens.new_empty((*tokens.shape, 3), dtype=torch.float32)
    _logprobs_fwd(logits, tokens, 0, logprobs, entropy, None, None, saved)
    return logprobs, entropy, saved


def token_logprobs_bwd(logits, tokens, saved, dlogprobs, dentropy=None, dlogits=None):
    """The gradient to the logits of L = sum(dlogprobs * logprobs) + sum(dentropy * entropy), on the current stream, in
    logits' dtype; saved: as token_logprobs_save returned it.  dlogits=logits writes it over them."""
    import torch
    given = () if dlogits is None else _given(dlogits)
    if dlogits is None:
        dlogits = torch.empty_like(logits, memory_format=torch.contiguous_format)
    _launch("token_logprobs_bwd", logits, logits, tokens, saved, dlogprobs, dentropy, dlogits)
    if given:
        _note_written(given)
    return dlogits


# ---------------------------------------------------------------------------------------- autograd
#
# An output that is not used has no gradient (None), which the library takes as 0 where it is not the main one; what an input
# that needs no gradient would have is not made where the library can leave it out.

def _dense(grad):
    return None if grad is None else grad.contiguous()


class RMSNormFunction:
    """torch.autograd wrapper of the RMS norm: RMSNormFunction.apply(x, weight, residual, eps) -> (out, residual_out),
    differentiable in x, weight and residual (residual may be None: residual_out is too).  Graph capture and
    derivatives: as for GatedScanFunction."""

    @staticmethod
    def apply(x, weight, residual=None, eps=1e-5):
        return _function("norm", _make_norm).apply(x, weight, residual, eps)


def _make_norm():
    import torch

    class _Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, residual, eps):
            out, stream, rstd = rms_norm_fwd_save(x, weight, residual=residual, eps=eps)
            ctx.save_for_backward(x if stream is None else stream, weight, rstd)
            ctx.set_materialize_grads(False)
            ctx.dtype = x.dtype
            return out, stream

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dout, dstream):
            z, weight, rstd = ctx.saved_tensors
            dout = z.new_zeros(z.shape, dtype=ctx.dtype) if dout is None else dout.contiguous()
            g = rms_norm_bwd(z, weight, rstd, dout, dresidual_out=_dense(dstream),
                             return_dresidual=ctx.needs_input_grad[2], return_dweight=ctx.needs_input_grad[1])
            return g["dx"], g.get("dweight"), g.get("dresidual"), None

    return _Norm


class LinearAttentionFunction:
    """torch.autograd wrapper of linear attention: LinearAttentionFunction.apply(q, k, v, rate, scale, initial_state,
    seq_lens) -> (out, last_state), differentiable in q, k, v and initial_state (scale, initial_state and seq_lens may
    be None).  rate is a constant: one that requires gradients is refused.  Decoding goes on from
    last_state.detach().clone().  Graph capture and derivatives: as for GatedScanFunction."""

    @staticmethod
    def apply(q, k, v, rate, scale=None, initial_state=None, seq_lens=None):
        if rate.requires_grad:
            raise ValueError("linear attention's decay has no gradient: pass a detached rate")
        return _function("attention", _make_attention).apply(q, k, v, rate, scale, initial_state, seq_lens)


def _aligned(t):
    """t (dense, or None) 16-byte aligned: a gradient that autograd delivers may be a view of another at any element."""
    return t.clone() if t is not None and t.data_ptr() % 16 else t


def _make_attention():
    import torch

    class _Attention(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, rate, scale, initial_state, seq_lens):
            out, last = linear_attention_fwd(q, k, v, rate, scale=scale, initial_state=initial_state, seq_lens=seq_lens)
            ctx.save_for_backward(q, k, v, rate, initial_state, seq_lens)
            ctx.set_materialize_grads(False)
            ctx.scale, ctx.shape = scale, out.shape
            return out, last

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dout, dlast):
            q, k, v, rate, initial_state, seq_lens = ctx.saved_tensors
            dout = q.new_zeros(ctx.shape) if dout is None else _aligned(dout.contiguous())
            g = linear_attention_bwd(q, k, v, rate, dout, scale=ctx.scale, initial_state=initial_state,
                                     seq_lens=seq_lens, dlast_state=_aligned(_dense(dlast)),
                                     return_dinitial_state=ctx.needs_input_grad[5])
            return g["dq"], g["dk"], g["dv"], None, None, g.get("dinitial_state"), None

    return _Attention


class TokenLogprobsFunction:
    """torch.autograd wrapper of token_logprobs: TokenLogprobsFunction.apply(logits, tokens) -> (logprobs, entropy),
    differentiable in logits.  Graph capture and derivatives: as for GatedScanFunction."""

    @staticmethod
    def apply(logits, tokens):
        return _function("logprobs", _make_logprobs).apply(logits, tokens)


def _make_logprobs():
    import torch

    class _Logprobs(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, tokens):
            logprobs, entropy, saved = token_logprobs_save(logits, tokens)
            ctx.save_for_backward(logits, tokens, saved)
            ctx.set_materialize_grads(False)
            return logprobs, entropy

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dlogprobs, dentropy):
            logits, tokens, saved = ctx.saved_tensors
            if dlogprobs is None:
                dlogprobs = saved.new_zeros(tokens.shape)
            return token_logprobs_bwd(logits, tokens, saved, dlogprobs.contiguous(), _dense(dentropy)), None

    return _Logprobs


# ------------------------------------------------------------------------------------- bound steps

class _Bound:
    """A library function bound to descriptors of tensors that it keeps alive; `args` places tensors and numbers."""

    def _bind(self, name, args, written, stream):
        import torch
        self._name, self._written = name, [t for t in written if t is not None]
        self._keep = args
        self._descs = [_desc(t) if isinstance(t, torch.Tensor) else t for t in args]
        self._args = tuple(ctypes.byref(d) if isinstance(d, ctypes.Structure) else d for d in self._descs) + (stream,)
        self._fn = getattr(load_library(), name)

    def _call(self):
        st = self._fn(*self._args)
        if st != 0:
            raise MssError(st, self._name)
        _note_written(self._written)


class RMSNormStep(_Bound):
    """mss_rms_norm_fwd bound to fixed device buffers, for decode loops: descriptors and stream are taken once, here.
    Arguments as for rms_norm_fwd; calling it updates `residual` (when given) in place and writes `out` (returned)."""

    def __init__(self, x, weight, residual=None, eps=1e-5, out=None, stream=None):
        _refuse_written(residual, out)
        _same_device(x, (weight, residual, out))
        stream = _bound_stream(x, stream)
        self.out = _empty_on(stream, x.shape, x.dtype, x.device) if out is None else out
        self._bind("mss_rms_norm_fwd", (x, residual, weight, float(eps), self.out, residual, None, None),
                   (residual, self.out), stream)

    def __call__(self):
        self._call()
        return self.out


class LinearAttentionUpdateStep(_Bound):
    """mss_linear_attention_update bound to fixed device buffers, for decode loops that refill the same input buffers
    every token.  Arguments as for linear_attention_update; calling it updates `state` in place and writes `out`
    (returned)."""

    def __init__(self, state, q, k, v, rate, scale=None, out=None, stream=None):
        _refuse_written(state, out)
        _same_device(q, (state, k, v, rate, out))
        stream = _bound_stream(q, stream)
        if out is None:
            out = _empty_on(stream, (q.shape[0], rate.shape[0], v.shape[-1]), q.dtype, q.device)
        self.out = out
        self._bind("mss_linear_attention_update", (state, q, k, v, rate, _scale_of(scale, q), out), (state, out), stream)

    def __call__(self):
        self._call()
        return self.out
