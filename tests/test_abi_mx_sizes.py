"""Refusals of the MXFP4 entry points at sizes whose rounding up would pass 31 bits,
without a GPU: they come before any device work."""

import ctypes

import pytest

import __graft_entry__
from nvfp4_block_scaled_topk_gb300 import megamoe

F = ctypes.c_void_p(256)  # an aligned address that is never touched
SHAPE = 2
TOO_MANY = [1 << 30, (1 << 31) - 32]


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return megamoe.load()


@pytest.mark.parametrize("n", TOO_MANY)
def test_columns(lib, n):
    for transpose in (0, 1):
        assert lib.megamoe_quantize_mxfp4(F, 0, 1, n, n, transpose, F, F, 0, None, None) == SHAPE
    for K, N in ((n, 32), (32, n)):
        assert lib.megamoe_linear_mxfp4(F, 0, 1, K, K, F, F, N, 2, F, N, F, 1 << 62, None) == SHAPE
        assert lib.megamoe_linear_mxfp4_backward(F, 0, N, F, 0, K, F, 0, K, 1, K, N, F, 2, K, F, 2, K,
                                                 F, 1 << 62, None) == SHAPE
