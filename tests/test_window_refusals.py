"""Refusals of the window's operators at the ends of their arguments, on a machine without a GPU."""
import ctypes

import pytest

import verify_weight_streaming_b200 as mr

A = ctypes.c_void_p(256)


@pytest.mark.parametrize("inter,code", [
    (2 ** 30, mr.MR_ERR_UNSUPPORTED), (2 ** 31 - 64, mr.MR_ERR_UNSUPPORTED), (2 ** 30 - 64, mr.MR_ERR_UNSUPPORTED),
    (2 ** 20 + 64, mr.MR_ERR_UNSUPPORTED), (-64, mr.MR_ERR_INVALID_ARG), (-(2 ** 31), mr.MR_ERR_INVALID_ARG),
    (-(2 ** 30), mr.MR_ERR_INVALID_ARG),
])
def test_moe_window_w4_inter(inter, code):
    """2 * inter is formed only for sizes that hold it."""
    assert mr.lib.moe_window_w4(A, 128, A, A, 4, A, 1 << 62, A, 1 << 62, A, 128, 2, 4, 8, 128, inter, 0, 64, mr.MR_F32, 0,
                                A, 1 << 62, None) == code
