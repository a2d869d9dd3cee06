"""The RMS norm, linear attention and token log probabilities without a GPU: every invalid call is refused with its
documented status before any HIP call (the device addresses below are made up), calls with nothing to do return, and the
scratch queries look at sizes alone."""
import ctypes
import os

import pytest

import selective_state_space_06_amd as mss
from selective_state_space_06_amd import MSS_BF16, MSS_F32, MSS_F8E4M3, MSS_I32, Tensor

OK, NULL_ARG, SHAPE, DTYPE, LAYOUT, ALIAS, UNSUPPORTED = 0, -1, -2, -3, -4, -5, -6
_next = [0x10000000]


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(mss.LIB_PATH):
        from selective_state_space_06_amd import build
        build.build()
    return mss.load_library()


def T(shape, dtype=MSS_F32):
    n = 4
    for s in shape:
        n *= max(1, s)
    a = _next[0]
    _next[0] += (n + 0xFFFF) & ~0xFFFF
    return Tensor.make(a, dtype, shape)


def shape_of(t):
    return list(t.shape)[:t.ndim]


def moved(t, nbytes):
    return Tensor.make(t.data + nbytes, t.dtype, shape_of(t))


def strided(t):
    s = shape_of(t)
    st, acc = [], 2
    for e in reversed(s):
        st.insert(0, acc)
        acc *= e
    return Tensor.make(t.data, t.dtype, s, st)


B, L, W, H, Q, KH, VH, K, V, NV = 2, 70, 300, 8, 2, 4, 8, 32, 48, 70000


def norm_args(dt=MSS_BF16):
    return dict(x=T([B, L, W], dt), residual=T([B, L, W]), weight=T([W]), eps=1e-5, out=T([B, L, W], dt),
                residual_out=T([B, L, W]), rstd=T([B, L]), scales=None)


def e4m3_args(dt=MSS_BF16):
    return dict(norm_args(dt), out=T([B, L, W], MSS_F8E4M3), scales=T([B, L, 3]))


def norm_bwd_args(dt=MSS_BF16):
    return dict(z=T([B, L, W]), weight=T([W]), rstd=T([B, L]), dout=T([B, L, W], dt), dresidual_out=T([B, L, W]),
                dx=T([B, L, W], dt), dresidual=T([B, L, W]), dweight=T([W]), scratch=T([1 << 20]))


def attn_args(dt=MSS_BF16):
    return dict(q=T([B, L, Q, K], dt), k=T([B, L, KH, K], dt), v=T([B, L, VH, V], dt), rate=T([H]), scale=0.5,
                initial_state=T([B, H, K, V]), seq_lens=T([B], MSS_I32), out=T([B, L, H, V], dt),
                last_state=T([B, H, K, V]), scratch=T([1 << 20]))


def attn_bwd_args(dt=MSS_BF16):  # eight heads to a query: their gradients meet in scratch
    return dict(q=T([B, L, Q, K], dt), k=T([B, L, KH, K], dt), v=T([B, L, VH, V], dt), rate=T([2 * H]), scale=0.5,
                initial_state=T([B, 2 * H, K, V]), seq_lens=T([B], MSS_I32), dout=T([B, L, 2 * H, V], dt),
                dlast_state=T([B, 2 * H, K, V]), dq=T([B, L, Q, K], dt), dk=T([B, L, KH, K], dt), dv=T([B, L, VH, V], dt),
                dinitial_state=T([B, 2 * H, K, V]), scratch=T([1 << 20]))


def step_args(dt=MSS_BF16):
    return dict(state=T([B, H, K, V]), q=T([B, Q, K], dt), k=T([B, KH, K], dt), v=T([B, VH, V], dt), rate=T([H]),
                scale=0.5, out=T([B, H, V], dt))


def logprob_args(dt=MSS_BF16):
    return dict(logits=T([B, L, NV], dt), tokens=T([B, L], MSS_I32), logprobs=T([B, L]), entropy=T([B, L]),
                top_logprobs=T([B, L, 5]), top_tokens=T([B, L, 5], MSS_I32), saved=T([B, L, 3]), scratch=T([1 << 20]))


def logprob_bwd_args(dt=MSS_BF16):
    return dict(logits=T([B, L, NV], dt), tokens=T([B, L], MSS_I32), saved=T([B, L, 3]), dlogprobs=T([B, L]),
                dentropy=T([B, L]), dlogits=T([B, L, NV], dt))


CALLS = {"norm": (norm_args, mss.rms_norm_fwd_raw), "e4m3": (e4m3_args, mss.rms_norm_fwd_raw),
         "norm_bwd": (norm_bwd_args, mss.rms_norm_bwd_raw), "attn": (attn_args, mss.linear_attention_fwd_raw),
         "attn_bwd": (attn_bwd_args, mss.linear_attention_bwd_raw), "step": (step_args, mss.linear_attention_update_raw),
         "logprob": (logprob_args, mss.token_logprobs_fwd_raw),
         "logprob_bwd": (logprob_bwd_args, mss.token_logprobs_bwd_raw)}
REQUIRED = {"norm": "x residual weight out residual_out", "e4m3": "x weight out scales",
            "norm_bwd": "z weight rstd dout dx scratch", "attn": "q k v rate out",
            "attn_bwd": "q k v rate dout dq dk dv scratch", "step": "state q k v rate out",
            "logprob": "logits tokens logprobs top_logprobs top_tokens scratch",
            "logprob_bwd": "logits tokens saved dlogprobs dlogits"}
OUTPUTS = {"norm": "out residual_out rstd", "e4m3": "out residual_out rstd scales",
           "norm_bwd": "dx dresidual dweight scratch", "attn": "out last_state",
           "attn_bwd": "dq dk dv dinitial_state scratch", "step": "state out",
           "logprob": "logprobs entropy top_logprobs top_tokens saved scratch", "logprob_bwd": "dlogits"}


ALIGNED = {"attn": "q k v initial_state out last_state", "step": "state",
           "attn_bwd": "q k v initial_state dout dlast_state dq dk dv dinitial_state"}


def call(op, a):
    return CALLS[op][1](*a.values(), None)


def each(names):
    return [(op, n) for op, ns in names.items() for n in ns.split()]


@pytest.mark.parametrize("op,name", each(REQUIRED))
def test_null_required(op, name):
    a = CALLS[op][0]()
    a[name] = None
    assert call(op, a) == NULL_ARG
    a = CALLS[op][0]()
    a[name].data = None
    assert call(op, a) == NULL_ARG


@pytest.mark.parametrize("op", CALLS)
def test_shape_dtype_layout_of_every_tensor(op):
    for name, t in CALLS[op][0]().items():
        if not isinstance(t, Tensor):
            continue
        shape = shape_of(t)
        # scratch that these sizes do not need has no least size
        for j in range(0 if (op, name) == ("attn", "scratch") else t.ndim):
            a = CALLS[op][0]()
            bad = list(shape)
            bad[j] = 1 if name == "scratch" else bad[j] + 1
            if (op, name, j) in (("logprob", "logits", 2),):
                continue  # the vocabulary stands in no other shape
            a[name] = Tensor.make(t.data, t.dtype, bad)
            assert call(op, a) == SHAPE, (op, name, j)
        a = CALLS[op][0]()
        a[name] = Tensor.make(t.data, t.dtype, shape + [1] if t.ndim < 4 else shape[1:])
        assert call(op, a) == SHAPE, (op, name, "ndim")
        a = CALLS[op][0]()
        a[name] = Tensor.make(t.data, t.dtype, [-1] + shape[1:])
        assert call(op, a) == SHAPE, (op, name, "negative")
        for dt in (MSS_F32, MSS_BF16, MSS_I32, MSS_F8E4M3, 7):
            a = CALLS[op][0]()
            if dt == a[name].dtype:
                continue
            if (op, name, dt) in (("logprob", "logits", MSS_F32), ("e4m3", "x", MSS_F32)):  # types that stand alone
                continue
            a[name].dtype = dt
            # an 8-bit output without scales lacks them
            want = NULL_ARG if (op, name, dt) == ("norm", "out", MSS_F8E4M3) else DTYPE
            assert call(op, a) == want, (op, name, dt)
        a = CALLS[op][0]()
        a[name] = strided(a[name])
        assert call(op, a) == LAYOUT, (op, name)
        if t.dtype != MSS_F8E4M3:
            a = CALLS[op][0]()
            a[name] = moved(a[name], 1)
            assert call(op, a) == LAYOUT, (op, name)


@pytest.mark.parametrize("op,name", each(ALIGNED))
def test_sixteen_byte_alignment(op, name):
    a = CALLS[op][0]()
    a[name] = moved(a[name], 8)
    assert call(op, a) == LAYOUT


@pytest.mark.parametrize("op,name", each(OUTPUTS))
def test_overlaps_are_refused(op, name):
    for other, t in CALLS[op][0]().items():
        if other == name or not isinstance(t, Tensor):
            continue
        if (name, other) in (("residual_out", "residual"), ("dlogits", "logits")):
            continue  # in place: allowed, and tested where it runs
        a = CALLS[op][0]()
        a[name].data = a[other].data
        assert call(op, a) == ALIAS, (op, name, other)


def test_partial_overlaps_in_place_are_refused():
    a = norm_args()
    a["residual_out"].data = a["residual"].data + 4 * W
    assert call("norm", a) == ALIAS
    a = logprob_bwd_args()
    a["dlogits"].data = a["logits"].data + 2 * NV
    assert call("logprob_bwd", a) == ALIAS


def test_norm_scales_and_widths():
    for parts, want in ((1, None), (3, None), (2, SHAPE), (4, SHAPE), (0, SHAPE)):
        a = e4m3_args()
        a["scales"] = T([B, L, parts])
        a["rstd"] = T([B, L + 1]) if want is None else a["rstd"]  # the next refusal: the scales were in order
        assert call("e4m3", a) == SHAPE
        if want is None:
            a = e4m3_args()
            a["scales"] = T([B, L, parts])
            a["out"].dtype = MSS_BF16
            assert call("e4m3", a) == DTYPE
    a = norm_args()
    a["scales"] = T([B, L, 3])
    assert call("norm", a) == DTYPE
    for t in ("residual", "residual_out"):
        a = norm_args()
        a[t] = None
        assert call("norm", a) == NULL_ARG
    wide = {n: T([2, 16385] if t.ndim == 3 else [2] if n == "rstd" else [16385], t.dtype) if isinstance(t, Tensor) else t
            for n, t in norm_args().items()}
    assert call("norm", wide) == UNSUPPORTED
    wide = {n: T([2, 16385] if t.ndim == 3 else [2] if n == "rstd" else [16385], t.dtype)
            for n, t in norm_bwd_args().items()}
    assert call("norm_bwd", wide) == UNSUPPORTED
    flat = {n: T([W], t.dtype) if isinstance(t, Tensor) else t for n, t in norm_args().items()}
    assert call("norm", flat) == SHAPE


def test_attention_heads_and_dims():
    for name, n in (("q", 3), ("k", 16), ("v", 5)):
        a = attn_args()
        s = shape_of(a[name])
        a[name] = T([B, L, n, s[3]], MSS_BF16)
        assert call("attn", a) == SHAPE
    for kd, vd in ((24, 48), (32, 40), (144, 48), (32, 256)):
        a = dict(q=T([B, L, Q, kd], MSS_BF16), k=T([B, L, KH, kd], MSS_BF16), v=T([B, L, VH, vd], MSS_BF16), rate=T([H]),
                 scale=1.0, initial_state=None, seq_lens=None, out=T([B, L, H, vd], MSS_BF16), last_state=None,
                 scratch=None)
        assert call("attn", a) == UNSUPPORTED
        s = dict(state=T([B, H, kd, vd]), q=T([B, Q, kd]), k=T([B, KH, kd]), v=T([B, VH, vd]), rate=T([H]), scale=1.0,
                 out=T([B, H, vd]))
        assert call("step", s) == UNSUPPORTED
    none = dict(q=T([B, L, 1, K]), k=T([B, L, 1, K]), v=T([B, L, 1, V]), rate=Tensor.make(0, MSS_F32, [0]), scale=1.0,
                initial_state=None, seq_lens=None, out=Tensor.make(0, MSS_F32, [B, L, 0, V]), last_state=None,
                scratch=None)
    assert call("attn", none) == SHAPE


def test_logprob_limits():
    a = logprob_args()
    a.update(top_logprobs=T([B, L, 65]), top_tokens=T([B, L, 65], MSS_I32))
    assert call("logprob", a) == UNSUPPORTED
    a = logprob_args()
    a.update(top_logprobs=T([B, L, 0]), top_tokens=T([B, L, 0], MSS_I32))
    assert call("logprob", a) == SHAPE
    a = logprob_args()
    a["logits"] = Tensor.make(0, MSS_BF16, [B, L, 0])
    assert call("logprob", a) == SHAPE


def test_scratch_queries():
    assert mss.rms_norm_bwd_scratch(8192, 2560) >= 2560
    assert mss.rms_norm_bwd_scratch(0, 7) >= 0
    assert all(n >= 0 for n in mss.linear_attention_scratch(1, 32768, 16, 16, 4, 4, 64, 64))
    assert mss.linear_attention_scratch(4, 2048, 80, 8, 8, 80, 128, 64)[1] >= 4 * 2048 * 80 * 128  # partial sums
    assert mss.token_logprobs_scratch(0, 5, 0) == 0
    for f, args, want in ((mss.rms_norm_bwd_scratch, (-1, 4), SHAPE), (mss.rms_norm_bwd_scratch, (4, 0), SHAPE),
                          (mss.rms_norm_bwd_scratch, (4, 16385), UNSUPPORTED),
                          (mss.rms_norm_bwd_scratch, (1 << 45, 64), SHAPE),
                          (mss.linear_attention_scratch, (1, 5, 6, 4, 6, 6, 16, 16), SHAPE),
                          (mss.linear_attention_scratch, (1, 5, 6, 6, 6, 6, 20, 16), UNSUPPORTED),
                          (mss.linear_attention_scratch, (1 << 40, 5, 6, 6, 6, 6, 16, 16), UNSUPPORTED),
                          (mss.linear_attention_scratch, (1, 1 << 31, 1, 1, 1, 1, 16, 16), UNSUPPORTED),
                          (mss.linear_attention_scratch, (1, 5, 32769, 1, 1, 1, 16, 16), UNSUPPORTED),
                          (mss.linear_attention_scratch, (1 << 15, 5, 64, 1, 1, 1, 16, 16), UNSUPPORTED),
                          (mss.linear_attention_scratch, (1, -1, 6, 6, 6, 6, 16, 16), SHAPE),
                          (mss.token_logprobs_scratch, (4, 0, 1), SHAPE), (mss.token_logprobs_scratch, (4, 9, 65), UNSUPPORTED),
                          (mss.token_logprobs_scratch, (4, 1 << 31, 0), UNSUPPORTED)):
        with pytest.raises(mss.MssError) as e:
            f(*args)
        assert e.value.status == want, (f.__name__, args)
    lib, n = mss.load_library(), ctypes.c_int64()
    assert lib.mss_rms_norm_bwd_scratch(1, 1, None) == NULL_ARG
    assert lib.mss_linear_attention_scratch(1, 1, 1, 1, 1, 1, 16, 16, None, ctypes.byref(n)) == NULL_ARG
    assert lib.mss_token_logprobs_scratch(1, 1, 1, None) == NULL_ARG


@pytest.mark.parametrize("op", CALLS)
def test_empty_batch_is_ok(op):
    a = CALLS[op][0]()
    for n, t in a.items():
        if isinstance(t, Tensor) and n not in ("scratch", "rate", "weight", "dweight"):
            a[n] = Tensor.make(0, t.dtype, [0] + shape_of(t)[1:])
    if op == "norm_bwd":  # the sum over no rows is still written
        a["dweight"] = None
    assert call(op, a) == OK


HOST = {
    "rms_norm_fwd": lambda t, i: mss.rms_norm_fwd(t(3, 8), t(8)),
    "rms_norm_fwd_e4m3": lambda t, i: mss.rms_norm_fwd_e4m3(t(3, 8), t(8)),
    "rms_norm_bwd": lambda t, i: mss.rms_norm_bwd(t(3, 8), t(8), t(3), t(3, 8)),
    "linear_attention_fwd": lambda t, i: mss.linear_attention_fwd(*[t(1, 4, 2, 16)] * 3, t(2)),
    "linear_attention_bwd": lambda t, i: mss.linear_attention_bwd(*[t(1, 4, 2, 16)] * 3, t(2), t(1, 4, 2, 16)),
    "linear_attention_update": lambda t, i: mss.linear_attention_update(t(1, 2, 16, 16), *[t(1, 2, 16)] * 3, t(2)),
    "token_logprobs": lambda t, i: mss.token_logprobs(t(3, 8), i(3)),
    "token_logprobs_bwd": lambda t, i: mss.token_logprobs_bwd(t(3, 8), i(3), t(3, 3), t(3)),
    "RMSNormStep": lambda t, i: mss.RMSNormStep(t(3, 8), t(8)),
    "LinearAttentionUpdateStep": lambda t, i: mss.LinearAttentionUpdateStep(t(1, 2, 16, 16), *[t(1, 2, 16)] * 3, t(2)),
}


@pytest.mark.parametrize("name", HOST)
def test_front_end_refuses_host_tensors(name):
    import torch
    with pytest.raises(ValueError, match="device"):
        HOST[name](lambda *s: torch.zeros(s), lambda *s: torch.zeros(s, dtype=torch.int32))


WRITTEN = {
    "rms_norm_fwd": lambda s, t: mss.rms_norm_fwd(t(3, 8), t(8), out=s),
    "rms_norm_fwd residual": lambda s, t: mss.rms_norm_fwd(t(3, 8), t(8), residual=s, residual_out=s),
    "rms_norm_fwd_e4m3": lambda s, t: mss.rms_norm_fwd_e4m3(t(3, 8), t(8), residual=s, residual_out=s),
    "rms_norm_fwd_save": lambda s, t: mss.rms_norm_fwd_save(t(3, 8), t(8), rstd=s),
    "linear_attention_fwd": lambda s, t: mss.linear_attention_fwd(*[t(1, 4, 2, 16)] * 3, t(2), last_state=s),
    "linear_attention_update": lambda s, t: mss.linear_attention_update(s, *[t(1, 2, 16)] * 3, t(2)),
    "token_logprobs_bwd": lambda s, t: mss.token_logprobs_bwd(s, t(3), t(3, 3), t(3), dlogits=s),
    "RMSNormStep": lambda s, t: mss.RMSNormStep(t(3, 8), t(8), residual=s),
    "LinearAttentionUpdateStep": lambda s, t: mss.LinearAttentionUpdateStep(s, *[t(1, 2, 16)] * 3, t(2)),
}


@pytest.mark.parametrize("name", WRITTEN)
def test_written_tensors_that_require_gradients_are_refused(name):
    import torch
    leaf = torch.zeros(3, 8, requires_grad=True)
    for s in (leaf, leaf * 2):
        with pytest.raises(ValueError, match="gradient"):
            WRITTEN[name](s, lambda *n: torch.zeros(n))


def test_front_end_refusals():
    import torch
    t = torch.zeros
    with pytest.raises(ValueError, match="group"):
        mss.rms_norm_fwd_e4m3(t(3, 8), t(8), group=64)
    with pytest.raises(ValueError, match="decay"):
        mss.LinearAttentionFunction.apply(*[t(1, 4, 2, 16)] * 3, t(2, requires_grad=True))
