"""The RMS norm's eps is not negative: checked before any HIP call (a call without rows makes none).  No GPU."""
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


@pytest.mark.parametrize("eps,status", [(0.0, 0), (1e-5, 0), (float("inf"), 0), (-1e-5, -2), (float("-inf"), -2),
                                        (float("nan"), -2)])
def test_eps(eps, status):
    rows, weight = Tensor.make(0, MSS_F32, [0, 8]), Tensor.make(0x10000, MSS_F32, [8])
    assert mss.rms_norm_fwd_raw(rows, None, weight, eps, rows, None, None, None, None) == status
