"""GPU tests of what linear attention carries over many steps and out of large states, at slow and at fast decays, against
closed forms: with keys (or output gradients) of zeros a state only decays, and nothing later hides its error.

Tolerances relative to the result itself, u = 2^-24: with states, queries and values that are all positive no terms cancel.
  - a power l^n of at most 32 steps, or of a part's steps: exp2 and its correction 3 u; that product a rounding more.  A state
    after c chunks and p parts is (4 c + 4 p) u off: in powers themselves where l^n < 1/2, in l^n - 1 otherwise.
  - an output: three powers and their products 13 u; a sum of 16 products in three bf16 parts each, 48 u and 2^-25 for what
    the parts leave; the scale and the head's sum: 80 u with room.
  - a bf16 result half a step more, 2^-8.
Values under 2^-108 lose the last of their bf16 parts (under 2^-126, which the matrix cores take for 0): 16 terms of 2^-126 are
below 1e-35."""
import numpy as np
import pytest

from synth import round_to_bf16
from tests.gpu_helpers import dev, host64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
RATES = np.array([0.0, 1e-5, 0.01, 0.02, 0.3, 0.4, 0.5, 0.55, 0.7, 1.0, 2.0, 5.0], dtype=np.float32)


@pytest.fixture(scope="module")
def mss():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_06_amd as m
    m.load_library()
    return m


def close(got, ref, n, dtype, what):
    g = host64(got)
    lim = (n * U + (2.0 ** -8 if dtype == "bf16" else 0.0)) * np.abs(ref) + 1e-35
    assert g.shape == ref.shape and np.all(np.isfinite(g)), what
    bad = np.abs(g - ref) > lim
    assert not bad.any(), (what, np.argwhere(bad)[0], float(np.max(np.abs(g - ref) / lim)))


def check(mss, B, L, rate, dtype, K=16, V=16, size=1.0, lens=None, gradients=True):
    import torch
    H = len(rate)
    rng = np.random.default_rng(L + H)

    def draw(*s):
        a = rng.uniform(0.5, 1.5, s).astype(np.float32)
        return round_to_bf16(a) if dtype == "bf16" else a

    S = (size * rng.uniform(0.5, 1.5, (B, H, K, V))).astype(np.float32)
    E = (size * rng.uniform(0.5, 1.5, (B, H, K, V))).astype(np.float32)
    q, k, v, d = draw(B, L, H, K), draw(B, L, H, K), draw(B, L, H, V), draw(B, L, H, V)
    zk, zv, r = dev(np.zeros_like(k), dtype), dev(np.zeros_like(v), dtype), dev(rate)
    n = np.full(B, L) if lens is None else np.array(lens)
    dl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    t = np.arange(L)
    ok = (t < n[:, None])[..., None, None]
    steps = 4 * (L / 32 + L / 128 + 2)
    since = np.exp(-rate.astype(np.float64) * (t[:, None] + 1))[None, :, :, None]          # l^(t + 1)
    left = np.exp(-rate.astype(np.float64) * np.maximum(n[:, None, None] - 1 - t[:, None], 0))[..., None]  # l^(n - 1 - t)
    whole = np.exp(-rate.astype(np.float64) * n[:, None])[..., None, None]

    out, last = mss.linear_attention_fwd(dev(q, dtype), zk, zv, r, scale=0.5, initial_state=dev(S), seq_lens=dl)
    close(out, np.where(ok, 0.5 * since * np.einsum("blhk,bhkv->blhv", q.astype(np.float64), S), 0), steps + 80, dtype, "out")
    close(last, whole * S, steps + 8, "f32", "last_state")
    if not gradients:
        return
    g = mss.linear_attention_bwd(zk, dev(k, dtype), dev(v, dtype), r, zv, scale=0.5, initial_state=dev(S), seq_lens=dl,
                                 dlast_state=dev(E), return_dinitial_state=True)
    close(g["dinitial_state"], whole * E, steps + 8, "f32", "dinitial_state")
    close(g["dk"], np.where(ok, left * np.einsum("blhv,bhkv->blhk", v.astype(np.float64), E), 0), steps + 80, dtype, "dk")
    close(g["dv"], np.where(ok, left * np.einsum("blhk,bhkv->blhv", k.astype(np.float64), E), 0), steps + 80, dtype, "dv")
    g = mss.linear_attention_bwd(zk, zk, zv, r, dev(d, dtype), scale=0.5, initial_state=dev(S), seq_lens=dl)
    close(g["dq"], np.where(ok, 0.5 * since * np.einsum("blhv,bhkv->blhk", d.astype(np.float64), S), 0), steps + 80, dtype, "dq")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 31, 32, 33, 64, 100])
def test_carried_states(mss, L, dtype):
    check(mss, 2, L, RATES, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sequences_of_different_lengths(mss, dtype):
    check(mss, 5, 90, RATES, dtype, lens=[0, 1, 37, 64, 90])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K,V", [(128, 128), (64, 128), (128, 64)])
def test_large_states(mss, K, V, dtype):
    """More keys than 16 add up in as many more roundings: the limit's 80 u are for 16, and 128 are eight times the sum's 48."""
    rate = np.array([0.02, 0.3, 0.6], dtype=np.float32)
    import torch
    rng = np.random.default_rng(K)
    S = rng.uniform(0.5, 1.5, (1, 3, K, V)).astype(np.float32)
    q = round_to_bf16(rng.uniform(0.5, 1.5, (1, 70, 3, K)).astype(np.float32))
    z = torch.zeros(1, 70, 3, K, device="cuda"), torch.zeros(1, 70, 3, V, device="cuda")
    tt = torch.bfloat16 if dtype == "bf16" else torch.float32
    out, last = mss.linear_attention_fwd(dev(q, dtype), z[0].to(tt), z[1].to(tt), dev(rate), scale=0.5, initial_state=dev(S))
    t = np.arange(70)
    since = np.exp(-rate.astype(np.float64) * (t[:, None] + 1))[None, :, :, None]
    close(out, 0.5 * since * np.einsum("blhk,bhkv->blhv", q.astype(np.float64), S), 32 + 8 * 48, dtype, "out")
    close(last, np.exp(-rate.astype(np.float64) * 70)[:, None, None] * S, 24, "f32", "last_state")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1000, 2048, 12345])
def test_segments(mss, L, dtype):
    """One head in segments, few (their parts are added up where they are read) and many (joined by a kernel of their own)."""
    assert mss.linear_attention_scratch(1, L, 1, 1, 1, 1, 16, 16)[0] > 0
    for rate in (0.002, 0.006, 0.02, 0.03, 0.06):
        check(mss, 1, L, np.array([rate], dtype=np.float32), dtype, size=1e6)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_keys_before_a_pause(mss, dtype):
    """A few large keys, then zeros: what they left decays over the chunks and segments behind them."""
    import torch
    L, rate = 1500, np.array([0.004, 0.02, 0.05], dtype=np.float32)
    rng = np.random.default_rng(5)
    k, v = np.zeros((1, L, 3, 16), dtype=np.float32), np.zeros((1, L, 3, 16), dtype=np.float32)
    k[:, 3] = round_to_bf16((1e4 * rng.uniform(0.5, 1.5, (1, 3, 16))).astype(np.float32))
    v[:, 3] = round_to_bf16(rng.uniform(0.5, 1.5, (1, 3, 16)).astype(np.float32))
    q = round_to_bf16(rng.uniform(0.5, 1.5, (1, L, 3, 16)).astype(np.float32))
    out, last = mss.linear_attention_fwd(dev(q, dtype), dev(k, dtype), dev(v, dtype), dev(rate), scale=1.0)
    t = np.arange(L)
    gone = np.where(t[:, None] >= 3, np.exp(-rate.astype(np.float64) * (t[:, None] - 3)), 0.0)[None, :, :, None]
    qk = np.einsum("blhk,bhk->blh", q.astype(np.float64), k[:, 3])[..., None]
    n = 4 * (L / 32 + L / 128 + 2) + 80
    close(out, gone * qk * v[:, 3][:, None], n, dtype, "out")
    S = k[:, 3].astype(np.float64)[..., None] * v[:, 3][..., None, :]
    close(last, np.exp(-rate.astype(np.float64) * (L - 4))[:, None, None] * S, n, "f32", "last_state")
    assert torch.isfinite(out).all()


def test_one_token(mss):
    import torch
    rate = np.array([0.0, 1e-6, 0.1, 0.6, 0.8, 3.0, 9.0, 17.0, 40.0], dtype=np.float32)
    S = np.random.default_rng(1).uniform(0.5, 1.5, (3, 9, 16, 32)).astype(np.float32)
    state = dev(S)
    z = torch.zeros(3, 9, 16, device="cuda"), torch.zeros(3, 9, 32, device="cuda")
    q = torch.ones_like(z[0])
    for n in (1, 2):
        out = mss.linear_attention_update(state, q, z[0], z[1], dev(rate), scale=1.0)
        want = np.exp(-n * rate.astype(np.float64))[:, None, None] * S
        close(state, want, 4 * n, "f32", "state")
        close(out, want.sum(2), 4 * n + 24, "f32", "out")
