"""GPU tests of reordering's bounds (nothing beside a state is written) and of a bound beam search step's
refusals (before anything is written)."""
import numpy as np
import pytest

import oracle
from selective_state_space_06_amd import MssError
from tests.test_gated_gpu import mss  # noqa: F401

pytestmark = pytest.mark.gpu
SHAPE, DTYPE, LAYOUT, ALIAS, UNSUPPORTED = -2, -3, -4, -5, -6


# rows of 16, 8, 4 and 2 bytes' multiples, alone and many, that end inside a block of threads and at its end
@pytest.mark.parametrize("B,N", [(1, 1), (2, 4), (3, 5), (2, 8), (1, 16), (1, 17), (2, 32), (1, 33), (1, 64)])
@pytest.mark.parametrize("dtype,width", [("f32", 4), ("f32", 1024), ("f32", 4097), ("f32", 6), ("f32", 1), ("bf16", 8),
                                         ("bf16", 2), ("bf16", 1), ("bf16", 511), ("i32", 2052)])
@pytest.mark.parametrize("shift", [0, 1])
def test_reorder_writes_nothing_else(mss, B, N, dtype, width, shift):  # noqa: F811
    """Three states in one buffer with guards between them: every element outside the states keeps its value."""
    import torch
    t = {"f32": torch.float32, "bf16": torch.bfloat16, "i32": torch.int32}[dtype]
    rng = np.random.default_rng(B + N + width)
    n, guard = B * N * width, 4096
    whole = torch.arange(3 * (n + guard) + guard + 8, device="cuda").to(torch.int64).remainder(251).to(t)
    states, want = [], whole.clone()
    parents = rng.integers(0, N, (B, N)).astype(np.int32)
    at = torch.from_numpy(oracle.beam_reorder(np.arange(B * N), parents)).cuda()
    for k in range(3):
        lo = guard + k * (n + guard) + shift
        states.append(whole[lo:lo + n].view(B * N, width))
        want[lo:lo + n] = want[lo:lo + n].view(B * N, width)[at].reshape(-1)
    mss.beam_reorder(states, torch.from_numpy(parents).cuda())
    assert torch.equal(whole, want)


def search(mss, states, **kw):  # noqa: F811
    import torch
    logits = torch.randn((2, 3, 50), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    scores = torch.tensor([[-1.0, -2.0, -3.0]] * 2, device="cuda")
    fin = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    given = dict(logits=logits, scores=scores, fin=fin)
    states = states(given) if callable(states) else states
    before = [v.clone() for v in (scores, fin, *states)]
    with pytest.raises((MssError, ValueError, TypeError)) as e:
        mss.BeamSearchStep(logits, scores, states, finished=fin, end_token=4, **kw)()
    torch.cuda.synchronize()
    for a, b in zip((scores, fin, *states), before):
        assert torch.equal(a, b), "a refused step has written"
    return e.value


def test_a_refused_step_has_written_nothing(mss):  # noqa: F811
    import torch
    z = lambda *s, **k: torch.ones(s, device="cuda", **k)  # noqa: E731
    good = z(6, 7)
    assert search(mss, [good, z(5, 7)]).status == SHAPE
    assert search(mss, [good, z(6, 7, dtype=torch.float64)]).status == DTYPE
    assert search(mss, [z(7, 6).t()]).status == LAYOUT
    assert search(mss, [good, good]).status == ALIAS
    assert search(mss, [good, good[2:]]).status in (SHAPE, ALIAS)
    # the step itself puts these in the beams' new order
    assert search(mss, lambda g: [g["scores"].view(6)]).status == ALIAS
    assert search(mss, lambda g: [g["fin"].view(6)]).status == ALIAS
    assert search(mss, lambda g: [g["logits"].view(6, 50)]).status == ALIAS


def test_a_step_is_bound_without_touching_anything(mss):  # noqa: F811
    import torch
    logits, scores = torch.randn((2, 3, 50), device="cuda"), torch.zeros((2, 3), device="cuda")
    states = [torch.randn((6, 9), device="cuda"), torch.randn((6, 3), device="cuda").to(torch.bfloat16)]
    before = [v.clone() for v in (logits, scores, *states)]
    step = mss.BeamSearchStep(logits, scores, states)
    assert all(torch.equal(a, b) for a, b in zip((logits, scores, *states), before))
    parents, tokens = step()
    want = [torch.from_numpy(oracle.beam_reorder(np.arange(6), parents.cpu().numpy())).cuda()]
    assert all(torch.equal(a, b[want[0]]) for a, b in zip(states, before[2:]))
    empty = mss.BeamSearchStep(torch.empty((0, 3, 5), device="cuda"), torch.empty((0, 3), device="cuda"),
                               [torch.empty((0, 4), device="cuda")])
    assert empty()[0].shape == (0, 3)
    alone = mss.BeamSearchStep(logits, scores, [])
    assert alone()[1].shape == (2, 3)
