"""Workspaces of the 8-bit linear on both sides of the limits between its ways: dots keep a
status word only, few tokens their integers as bytes, more of them as fp16."""

import ctypes

import pytest

import __graft_entry__
from nvfp4_block_scaled_topk_gb300 import megamoe

MB = 1 << 20
SMALL = 3


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return megamoe.load()


def up(n):
    return (n + 255) // 256 * 256


@pytest.mark.parametrize("T,most", [(1, 98304), (2, 49152), (3, 24576), (4, 24576)])
def test_dots(lib, T, most):
    size = lib.megamoe_linear_int8_workspace_size
    for N in (8, 2048):
        assert size(T, 16, N) == size(T, most, N) == 256
        assert size(T, most + 16, N) >= 256 + up(4 * T + 256) + 2 * T * (most + 16)


@pytest.mark.parametrize("T,most", [(5, 12160), (8, 12160), (9, 6016), (12, 6016), (16, 6016)])
def test_few(lib, T, most):
    size = lib.megamoe_linear_int8_workspace_size
    for N in (8, 2048):
        for K in (16, 4096, most):
            assert size(T, K, N) == 256 + up(4 * T + 256) + up(T * K)
        assert size(T, most + 16, N) >= 256 + up(4 * T + 256) + 2 * T * (most + 16)
    F = [ctypes.c_void_p(i * 64 * MB) for i in range(1, 6)]
    bytes_ = size(T, most, 2048)
    assert lib.megamoe_linear_int8(F[0], 0, T, most, most, None, F[1], F[2], 2048, 2, F[3], 2048, F[4],
                                   bytes_ - 1, None) == SMALL


def test_more(lib):
    size = lib.megamoe_linear_int8_workspace_size
    assert size(17, 16, 8) == 256 + up(4 * 17 + 256) + up(2 * 17 * 16)
    # shares of a sum, for either type of result
    assert size(17, 7168, 2048) >= 256 + up(4 * 17 + 256) + up(2 * 17 * 7168) + 2 * 4 * 17 * 2048
