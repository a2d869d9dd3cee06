"""The torch front end's own refusals, without a GPU."""
import pytest

import selective_state_space_06_amd as mss


def test_a_single_tensor_is_no_sequence_of_states():
    """Iterated over, a (rows, width) tensor is a sequence of rows; with as many columns as rows they would be
    taken for states, and their elements moved."""
    import torch
    square, parents = torch.zeros(4, 4), torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(TypeError, match="sequence"):
        mss.beam_reorder(square, parents)
    with pytest.raises(TypeError, match="sequence"):
        mss.BeamSearchStep(torch.zeros(2, 2, 5), torch.zeros(2, 2), square)
    with pytest.raises(ValueError, match="device tensors"):  # the sequence is looked into
        mss.beam_reorder([square], parents)


def test_streams_without_torchs_private_call(monkeypatch):
    import torch

    from selective_state_space_06_amd import _recurrent
    monkeypatch.setattr(_recurrent, "_raw_stream_of", None)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: type("S", (), {"cuda_stream": 40 + index}))
    assert _recurrent._raw_stream()(2) == 42
