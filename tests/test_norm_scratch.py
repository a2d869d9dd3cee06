"""The RMS norm's backward without dweight looks at no scratch: whatever its descriptor holds.  No GPU: a call without rows
returns before any HIP call."""
import os

import pytest

import selective_state_space_06_amd as mss
from selective_state_space_06_amd import MSS_F32, Tensor


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(mss.LIB_PATH):
        from selective_state_space_06_amd import build
        build.build()
    return mss.load_library()


def test_scratch_that_is_not_needed_is_not_read():
    rows, flat = Tensor.make(0, MSS_F32, [0, 8]), Tensor.make(0x10000, MSS_F32, [8])
    scratch = Tensor.make(0x20000, MSS_F32, [4])
    scratch.ndim = 1 << 24  # far past the descriptor's own extents
    assert mss.rms_norm_bwd_raw(rows, flat, Tensor.make(0, MSS_F32, [0]), rows, None, rows, None, None, scratch, None) == 0
