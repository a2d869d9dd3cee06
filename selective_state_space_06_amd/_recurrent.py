"""Torch front end of the gated scan, the causal conv's gradients and beam search (argument
marshalling only, like _binding.py).

These entry points take their scratch from the caller.  The functions below take it from torch's
allocator on the current stream, so every call, and every captured graph, has its own; the bound
steps keep theirs.
"""
from __future__ import annotations

import ctypes

from ._binding import (
    MssError, Tensor, _bound_stream, _desc, _note_written, _ref, _refuse_written, load_library)

SAVED_SPACING = 512  # steps between two of gated_scan_fwd_save's states


# ------------------------------------------------------------------- raw calls (descriptors or None)

def gated_scan_scratch(batch, d_inner, L):
    """(floats of scratch mss_gated_scan_fwd needs, floats mss_gated_scan_bwd needs)."""
    st, fwd, bwd = _native().gated_scan_scratch(batch, d_inner, L)
    _raise(st, "mss_gated_scan_scratch")
    return fwd, bwd


def causal_conv1d_bwd_scratch(batch, d_inner, L, K):
    """Floats of scratch mss_causal_conv1d_bwd needs."""
    st, n = _native().causal_conv1d_bwd_scratch(batch, d_inner, L, K)
    _raise(st, "mss_causal_conv1d_bwd_scratch")
    return n


def beam_select_scratch(batch, beams, vocab, k):
    """Floats of scratch mss_beam_select needs."""
    st, n = _native().beam_select_scratch(batch, beams, vocab, k)
    _raise(st, "mss_beam_select_scratch")
    return n


def gated_scan_fwd_raw(x, fgate, igate, rate, initial_state, seq_lens, out, last_state, saved_states, scratch,
                       stream) -> int:
    return load_library().mss_gated_scan_fwd(_ref(x), _ref(fgate), _ref(igate), _ref(rate), _ref(initial_state),
                                             _ref(seq_lens), _ref(out), _ref(last_state), _ref(saved_states),
                                             _ref(scratch), stream)


def gated_scan_bwd_raw(x, fgate, igate, rate, seq_lens, saved_states, dout, dlast_state, dx, dfgate, digate, drate,
                       dinitial_state, scratch, stream) -> int:
    return load_library().mss_gated_scan_bwd(_ref(x), _ref(fgate), _ref(igate), _ref(rate), _ref(seq_lens),
                                             _ref(saved_states), _ref(dout), _ref(dlast_state), _ref(dx),
                                             _ref(dfgate), _ref(digate), _ref(drate), _ref(dinitial_state),
                                             _ref(scratch), stream)


def gated_state_update_raw(state, x, fgate, igate, rate, out, stream) -> int:
    return load_library().mss_gated_state_update(_ref(state), _ref(x), _ref(fgate), _ref(igate), _ref(rate),
                                                 _ref(out), stream)


def conv1d_bwd_raw(x, weight, bias, initial_state, silu_flag, dout, dfinal_state, dx, dweight, dbias,
                   dinitial_state, scratch, stream) -> int:
    return load_library().mss_causal_conv1d_bwd(_ref(x), _ref(weight), _ref(bias), _ref(initial_state),
                                                int(silu_flag), _ref(dout), _ref(dfinal_state), _ref(dx),
                                                _ref(dweight), _ref(dbias), _ref(dinitial_state), _ref(scratch),
                                                stream)


def beam_select_raw(logits, scores, finished, end_token, next_scores, parents, tokens, next_finished, scratch,
                    stream) -> int:
    return load_library().mss_beam_select(_ref(logits), _ref(scores), _ref(finished), int(end_token),
                                          _ref(next_scores), _ref(parents), _ref(tokens), _ref(next_finished),
                                          _ref(scratch), stream)


def beam_reorder_raw(states, parents, stream) -> int:
    return load_library().mss_beam_reorder(_pointers(states), len(states), _ref(parents), stream)


def _pointers(descs):
    """An array of pointers to descriptors (the caller keeps them alive)."""
    return (ctypes.POINTER(Tensor) * max(1, len(descs)))(*[ctypes.pointer(d) for d in descs])


# ------------------------------------------------------------------------------- torch front end

def _raise(status, where):
    if status != 0:
        raise MssError(status, where)


_native_module = None


def _native():
    """The `_native` module (built with the library, which load_library() has loaded first)."""
    global _native_module
    if _native_module is None:
        import torch
        load_library()
        try:
            from . import _native as m
        except ImportError as e:
            raise RuntimeError(f"the _native module is missing ({e}): build it with "
                               "`python -m selective_state_space_06_amd.build`") from e
        m.set_dtypes(torch.float32, torch.bfloat16, torch.int32, torch.float8_e4m3fn)
        _native_module = m
    return _native_module


_raw_stream_of = None


def _raw_stream():
    """The function from a device index to its current stream's handle: torch's own without the Stream object
    (1 us less a call), which is private to torch and may be absent."""
    global _raw_stream_of
    if _raw_stream_of is None:
        import torch
        _raw_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
    return _raw_stream_of


def _launch(name, x, *args):
    """The native call `name` on the current stream of x's device."""
    import torch
    fn = getattr(_native(), name)
    index = x.get_device()
    if index < 0:
        raise ValueError("libmamba_scan takes device tensors")
    stream = _raw_stream()(index)
    if index == torch.cuda.current_device():
        st = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            st = fn(*args, stream)
    if st != 0:
        raise MssError(st, "mss_" + name)


def _same_device(x, tensors):
    for t in tensors:
        if t is not None and t.get_device() != x.get_device():
            raise ValueError(f"libmamba_scan takes tensors of one device, got {x.device} and {t.device}")


def _scratch(floats, device):
    import torch
    return torch.empty(floats, dtype=torch.float32, device=device) if floats else None


def _gated_fwd(x, fgate, igate, rate, initial_state, seq_lens, out, last_state, saved_states):
    floats = gated_scan_scratch(*x.shape)[0] if x.ndim == 3 else 0
    _launch("gated_scan_fwd", x, x, fgate, igate, rate, initial_state, seq_lens, out, last_state, saved_states,
            _scratch(floats, x.device))


def _saved_like(x):
    import torch
    return torch.empty((x.shape[0], x.shape[1], -(-x.shape[2] // SAVED_SPACING)), dtype=torch.float32,
                       device=x.device)


def gated_scan_fwd(x, fgate, igate, rate, initial_state=None, seq_lens=None, return_last_state=True, out=None,
                   last_state=None):
    """Gated scan (mss_gated_scan_fwd) on the current stream of x's device: per channel
    h_t = a h_{t-1} + sqrt(1 - a^2) sigmoid(igate_t) x_t with a = exp(-rate sigmoid(fgate_t)), out = h.

    x, fgate, igate: (batch, d_inner, L) float32 or bfloat16 (the gates before their sigmoid); rate:
    (d_inner,) float32, positive and finite; initial_state: (batch, d_inner) float32 (None: zeros); seq_lens:
    (batch,) int32 on the device (None: all L; outputs past a sequence's end are 0).  Returns out (dtype
    of x), or (out, last_state) with last_state (batch, d_inner) float32."""
    import torch
    given = [t for t in (out, last_state) if t is not None]
    _refuse_written(*given)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    if return_last_state and last_state is None:
        last_state = torch.empty(x.shape[:2], dtype=torch.float32, device=x.device)
    _gated_fwd(x, fgate, igate, rate, initial_state, seq_lens, out, last_state if return_last_state else None, None)
    _note_written(given)
    return (out, last_state) if return_last_state else out


def gated_scan_fwd_save(x, fgate, igate, rate, initial_state=None, seq_lens=None, out=None, last_state=None,
                        saved_states=None):
    """gated_scan_fwd that also writes the states its backward starts from: saved_states
    (batch, d_inner, ceil(L / 512)) float32, the state entering every 512th step.  Returns
    (out, last_state, saved_states)."""
    import torch
    given = [t for t in (out, last_state, saved_states) if t is not None]
    _refuse_written(*given)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    if last_state is None:
        last_state = torch.empty(x.shape[:2], dtype=torch.float32, device=x.device)
    if saved_states is None:
        saved_states = _saved_like(x)
    _gated_fwd(x, fgate, igate, rate, initial_state, seq_lens, out, last_state, saved_states)
    _note_written(given)
    return out, last_state, saved_states


def gated_scan_bwd(x, fgate, igate, rate, dout, initial_state=None, seq_lens=None, dlast_state=None,
                   return_dinitial_state=False, saved_states=None):
    """Gradients of gated_scan_fwd for L = sum(dout * out) + sum(dlast_state * last_state), on the
    current stream.  Returns a dict: dx, dfgate, digate in x's dtype, drate (d_inner,) float32 and, with
    return_dinitial_state, dinitial_state (batch, d_inner) float32.
    saved_states: what gated_scan_fwd_save wrote for this forward (it carries the initial state); None:
    they are computed again here, from initial_state."""
    import torch
    if saved_states is None:
        saved_states = _saved_like(x)
        _gated_fwd(x, fgate, igate, rate, initial_state, seq_lens, None, None, saved_states)
    g = {n: torch.empty_like(x, memory_format=torch.contiguous_format) for n in ("dx", "dfgate", "digate")}
    g["drate"] = torch.empty_like(rate, memory_format=torch.contiguous_format)
    if return_dinitial_state:
        g["dinitial_state"] = torch.empty(x.shape[:2], dtype=torch.float32, device=x.device)
    floats = gated_scan_scratch(*x.shape)[1] if x.ndim == 3 else 0
    _launch("gated_scan_bwd", x, x, fgate, igate, rate, seq_lens, saved_states, dout, dlast_state, g["dx"],
            g["dfgate"], g["digate"], g["drate"], g.get("dinitial_state"), _scratch(floats, x.device))
    return g


def gated_state_update(state, x, fgate, igate, rate, out=None):
    """One token of the gated scan (mss_gated_state_update) on the current stream; `state`
    (batch, d_inner) float32 is updated in place.  x, fgate, igate: (batch, d_inner) float32 or
    bfloat16.  Returns out (batch, d_inner) in x's dtype."""
    import torch
    written = (state,) if out is None else (state, out)
    _refuse_written(*written)
    if out is None:
        out = torch.empty_like(x)
    _launch("gated_state_update", x, state, x, fgate, igate, rate, out)
    _note_written(written)
    return out


def causal_conv1d_bwd(x, weight, dout, bias=None, initial_state=None, silu=True, dfinal_state=None,
                      return_dinitial_state=False):
    """Gradients of causal_conv1d_fwd for L = sum(dout * out) + sum(dfinal_state * final_state), on the
    current stream.  Returns a dict: dx in x's dtype, dweight (d_inner, K), dbias (d_inner,) float32
    (also when bias is None) and, with return_dinitial_state, dinitial_state (batch, d_inner, K - 1) in
    x's dtype."""
    import torch
    g = dict(dx=torch.empty_like(x, memory_format=torch.contiguous_format),
             dweight=torch.empty_like(weight, memory_format=torch.contiguous_format),
             dbias=torch.empty(weight.shape[:1], dtype=torch.float32, device=x.device))
    if return_dinitial_state:
        g["dinitial_state"] = torch.empty((x.shape[0], x.shape[1], weight.shape[1] - 1), dtype=x.dtype,
                                          device=x.device)
    # shapes that the query refuses are refused by the call itself, with its own status
    ok = x.ndim == 3 and weight.ndim == 2 and 1 <= weight.shape[1] <= 4
    floats = causal_conv1d_bwd_scratch(*x.shape, weight.shape[1]) if ok else 0
    _launch("causal_conv1d_bwd", x, x, weight, bias, initial_state, 1 if silu else 0, dout, dfinal_state, g["dx"],
            g["dweight"], g["dbias"], g.get("dinitial_state"), _scratch(floats, x.device))
    return g


def beam_select(logits, scores, finished=None, end_token=None, k=None, next_scores=None, parents=None, tokens=None,
                next_finished=None):
    """The k best continuations (k: as many as there are beams) of every request's beams
    (mss_beam_select), on the current stream: by score + log softmax(logits), a finished beam going on
    with end_token alone at its own score.

    logits: (batch, beams, vocab) float32 or bfloat16; scores: (batch, beams) float32; finished:
    (batch, beams) int32, nonzero for a beam at its end (needs end_token).  Returns (next_scores
    float32, parents int32, tokens int32), each (batch, k), best first, and with `finished` given also
    next_finished int32.  next_scores=scores and next_finished=finished update those in place."""
    import torch
    given = [t for t in (next_scores, parents, tokens, next_finished) if t is not None]
    _refuse_written(*given)
    # outputs after the model of scores where they have its shape (empty_like takes half the time of empty)
    shape = (logits.shape[0], scores.shape[-1] if k is None else int(k))
    like = scores if scores.shape == shape else scores.new_empty(shape)
    if next_scores is None:
        next_scores = torch.empty_like(like, dtype=torch.float32)
    if parents is None:
        parents = torch.empty_like(like, dtype=torch.int32)
    if tokens is None:
        tokens = torch.empty_like(like, dtype=torch.int32)
    if next_finished is None and finished is not None:
        next_finished = torch.empty_like(like, dtype=torch.int32)
    ok = logits.ndim == 3 and 1 <= logits.shape[1] <= 64 and 1 <= shape[1] <= 64 and logits.shape[2] >= 1
    floats = beam_select_scratch(*logits.shape, shape[1]) if ok else 0
    _launch("beam_select", logits, logits, scores, finished, -1 if end_token is None else int(end_token), next_scores,
            parents, tokens, next_finished, _scratch(floats, logits.device))
    _note_written(given)
    got = (next_scores, parents, tokens)
    return got if next_finished is None else got + (next_finished,)


def _state_tuple(states):
    """The states as a tuple.  A tensor is refused: it would be taken for a sequence of its rows."""
    import torch
    if isinstance(states, torch.Tensor):
        raise TypeError("states is a sequence of tensors, got one tensor")
    return tuple(states)


def beam_reorder(states, parents):
    """Every state (batch * beams, ...) in place: row b * beams + j becomes the row of beam
    parents[b, j] (mss_beam_reorder), on the current stream.  states: a sequence of float32, bfloat16 or
    int32 tensors (all layers' scan states and conv windows in one call); parents: (batch, beams) int32;
    a parent outside [0, beams) leaves its row as it is.  Returns states."""
    given = _state_tuple(states)
    _refuse_written(*given)
    _launch("beam_reorder", parents, given, parents)
    _note_written(given)
    return states


# ---------------------------------------------------------------------------------------- autograd

_fns = {}


def _function(name, make):
    if name not in _fns:
        _fns[name] = make()
    return _fns[name]


class GatedScanFunction:
    """torch.autograd wrapper of the gated scan: GatedScanFunction.apply(x, fgate, igate, rate,
    initial_state, seq_lens) -> (out, last_state), differentiable in x, fgate, igate, rate and
    initial_state (initial_state, seq_lens may be None).  The forward keeps one state in 512 for the
    backward.  Decoding goes on from last_state.detach().clone(): the calls that write a state in place
    refuse one that requires gradients.  To capture a training step in a graph, capture
    gated_scan_fwd_save and gated_scan_bwd (tested); a captured backward() of this wrapper is untested.
    First derivatives in reverse mode only: no double backward, no forward mode, no vmap."""

    @staticmethod
    def apply(x, fgate, igate, rate, initial_state=None, seq_lens=None):
        return _function("gated", _make_gated).apply(x, fgate, igate, rate, initial_state, seq_lens)


def _make_gated():
    import torch

    class _Gated(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, fgate, igate, rate, initial_state, seq_lens):
            out, last, saved = gated_scan_fwd_save(x, fgate, igate, rate, initial_state=initial_state,
                                                   seq_lens=seq_lens)
            ctx.save_for_backward(x, fgate, igate, rate, seq_lens, saved)
            ctx.has_state = initial_state is not None
            return out, last

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dout, dlast):
            x, fgate, igate, rate, seq_lens, saved = ctx.saved_tensors
            g = gated_scan_bwd(x, fgate, igate, rate, dout.contiguous(), seq_lens=seq_lens,
                               dlast_state=dlast.contiguous(), return_dinitial_state=ctx.has_state,
                               saved_states=saved)
            return g["dx"], g["dfgate"], g["digate"], g["drate"], g.get("dinitial_state"), None

    return _Gated


class CausalConv1dFunction:
    """torch.autograd wrapper of the causal conv: CausalConv1dFunction.apply(x, weight, bias,
    initial_state, silu) -> (out, final_state), differentiable in x, weight, bias and initial_state
    (bias, initial_state may be None).  Graph capture: as for GatedScanFunction."""

    @staticmethod
    def apply(x, weight, bias=None, initial_state=None, silu=True):
        return _function("conv", _make_conv).apply(x, weight, bias, initial_state, silu)


def _make_conv():
    import torch

    from ._binding import causal_conv1d_fwd

    class _Conv(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, bias, initial_state, silu):
            out, final = causal_conv1d_fwd(x, weight, bias, initial_state=initial_state, silu=silu,
                                           return_final_state=True)
            ctx.save_for_backward(x, weight, bias, initial_state)
            ctx.silu = silu
            return out, final

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dout, dfinal):
            x, weight, bias, initial_state = ctx.saved_tensors
            g = causal_conv1d_bwd(x, weight, dout.contiguous(), bias=bias, initial_state=initial_state,
                                  silu=ctx.silu, dfinal_state=dfinal.contiguous(),
                                  return_dinitial_state=initial_state is not None)
            return (g["dx"], g["dweight"], g["dbias"] if bias is not None else None, g.get("dinitial_state"), None)

    return _Conv


# ------------------------------------------------------------------------------------- bound steps

def _empty_on(stream, shape, dtype, device, fill=None):
    """Memory whose earlier users are ordered before work on `stream` (a raw handle)."""
    import torch

    def make():
        return torch.empty(shape, dtype=dtype, device=device) if fill is None else \
            torch.full(shape, fill, dtype=dtype, device=device)

    with torch.cuda.device(device):
        if stream == torch.cuda.current_stream(device).cuda_stream:
            return make()
        with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device)):
            return make()


class GatedUpdateStep:
    """mss_gated_state_update bound to fixed device buffers, for decode loops that refill the same
    input buffers every token: descriptors and stream are taken once, here.  Arguments as for
    gated_state_update; calling it updates `state` in place and writes `out` (returned)."""

    def __init__(self, state, x, fgate, igate, rate, out=None, stream=None):
        _refuse_written(state, out)
        _same_device(x, (state, fgate, igate, rate, out))
        stream = _bound_stream(x, stream)
        self.out = _empty_on(stream, x.shape, x.dtype, x.device) if out is None else out
        self._keep = (state, x, fgate, igate, rate, self.out)
        self._descs = [_desc(t) for t in self._keep]
        self._args = tuple(_ref(d) for d in self._descs) + (stream,)
        self._fn = load_library().mss_gated_state_update

    def __call__(self):
        _raise(self._fn(*self._args), "mss_gated_state_update")
        _note_written((self._keep[0], self.out))
        return self.out


class BeamSearchStep:
    """One step of a beam search bound to fixed device buffers: mss_beam_select on `logits` with
    `scores` (and `finished`) updated in place, then mss_beam_reorder of `states` by the parents it
    chose.  Arguments as for beam_select and beam_reorder; calling it returns (parents, tokens), its own
    (batch, beams) int32 buffers, which the next call overwrites.  States that cannot be reordered, or that
    overlap logits, scores or finished, are refused here.  Without `finished` a beam that takes
    end_token goes on like any other."""

    def __init__(self, logits, scores, states, finished=None, end_token=None, stream=None):
        import torch
        states = _state_tuple(states)
        _refuse_written(scores, finished, *states)
        _same_device(logits, (scores, finished, *states))
        stream = _bound_stream(logits, stream)
        self.parents = _empty_on(stream, scores.shape, torch.int32, logits.device, fill=-1)
        self.tokens = _empty_on(stream, scores.shape, torch.int32, logits.device)
        floats = beam_select_scratch(*logits.shape, scores.shape[-1])
        scratch = _empty_on(stream, (floats,), torch.float32, logits.device)
        self._keep = (logits, scores, finished, self.parents, self.tokens, scratch, *states)
        self._written = [t for t in (scores, finished, self.parents, self.tokens, *states) if t is not None]
        lo, sc, fi, pa, to, scr, *sts = [_desc(t) for t in self._keep]
        self._descs = (lo, sc, fi, pa, to, scr, sts)
        self._select_args = (_ref(lo), _ref(sc), _ref(fi), -1 if end_token is None else int(end_token), _ref(sc),
                             _ref(pa), _ref(to), _ref(fi), _ref(scr), stream)
        self._reorder_args = (_pointers(sts), len(sts), _ref(pa), stream)
        self._lib = load_library()
        # What mss_beam_reorder refuses has to be refused before mss_beam_select has moved the scores: asked now, with
        # parents of -1, which leave every row as it is.  What the selection reads or writes is no state either.
        apart = [_desc(t.flatten(0, 1)) for t in (logits, scores, finished) if t is not None and t.ndim > 1]
        with torch.cuda.device(logits.device):
            st = self._lib.mss_beam_reorder(_pointers(sts + apart), len(sts) + len(apart), _ref(pa), stream)
        _raise(st, "mss_beam_reorder")

    def __call__(self):
        _raise(self._lib.mss_beam_select(*self._select_args), "mss_beam_select")
        _raise(self._lib.mss_beam_reorder(*self._reorder_args), "mss_beam_reorder")
        _note_written(self._written)
        return self.parents, self.tokens
