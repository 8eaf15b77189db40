"""Results of the 16-bit experts' operators and the 8-bit integer linear that have memory
in common with what the call reads, or with each other: refused, without a GPU."""

import ctypes

import pytest

import __graft_entry__
from nvfp4_block_scaled_topk_gb300 import megamoe

P = None
INVALID = 1
BF, F32, I8 = 0, 1, 3
MB = 1 << 20


def at(mb, more=0):
    """An address that is never touched; matrices of the calls below are under 64 KB."""
    return ctypes.c_void_p(mb * MB + more)


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return megamoe.load()


R, K, N, E = 40, 64, 72, 4


@pytest.mark.parametrize("change", [
    dict(out=at(1)), dict(out=at(1, 128)), dict(out=at(1, R * K * 2 - 16)), dict(x=at(4, (R - 1) * N * 2)),
    dict(out=at(2)), dict(out=at(2, E * N * K * 2 - 16)), dict(w=at(4, R * N * 2 - 16)),
    dict(out_type=F32, x=at(4, R * N * 2 + 512)),  # behind 16-bit results, not behind fp32 ones
    dict(ld_x=144, ld_out=144, out=at(1, 112)),  # a row's columns, one beyond the other's first
    dict(ld_x=144, ld_out=144, out=at(1, 160 + 288)),  # ... and into the next row's
    dict(ld_x=144, ld_out=152, out=at(1, 128))])
def test_grouped(lib, change):
    a = dict(x=at(1), type=BF, rows=R, ld_x=K, w=at(2), E=E, N=N, K=K, off=at(3), poff=P, out_type=BF,
             out=at(4), ld_out=N, status=P) | change
    assert lib.megamoe_grouped_linear(*a.values(), P) == INVALID


@pytest.mark.parametrize("change", [
    dict(gx=at(1)), dict(gx=at(2)), dict(gx=at(3)), dict(gx=at(6)), dict(gw=at(1)), dict(gw=at(2)),
    dict(gw=at(3)), dict(w_type=BF, gw=at(3)), dict(gw=at(5, 32)), dict(gx=at(2, 256)),
    dict(w=P, gx=P, gw=at(2)), dict(w=P, gx=P, gw=at(1)),  # grad_w alone reads both
    dict(x=P, gw=P, gx=at(3)), dict(x=P, gw=P, gx=at(1))])  # grad_x alone these
def test_grouped_backward(lib, change):
    a = dict(g=at(1), ld_g=N, x=at(2), ld_x=K, w=at(3), type=BF, rows=R, E=E, N=N, K=K, off=at(4), poff=P,
             gx=at(5), ld_gx=K, w_type=F32, gw=at(6), status=P) | change
    assert lib.megamoe_grouped_linear_backward(*a.values(), P) == INVALID


@pytest.mark.parametrize("change", [
    dict(out=at(1, 16)), dict(out=at(1, 128 + 16)), dict(out=at(1), ld_out=64), dict(out=at(1, 256)),
    dict(a=at(2, 3 * 64 * 2))])
def test_silu(lib, change):
    a = dict(a=at(1), type=BF, rows=4, I=64, ld_a=128, live=P, out=at(2), ld_out=64)
    if "ld_out" not in change:
        a["ld_out"] = 128  # the stride of a, at other columns or rows
    assert lib.megamoe_silu_mul(*(a | change).values(), P) == INVALID


@pytest.mark.parametrize("change", [
    dict(ga=at(2, 16)), dict(ga=at(2, 128)), dict(ga=at(2), ld_ga=136), dict(ga=at(1)),
    dict(ga=at(1), ld_g=128, g=at(1, 64)), dict(ga=at(1, 256), ld_g=128)])
def test_silu_backward(lib, change):
    a = dict(g=at(1), ld_g=64, a=at(2), type=BF, rows=4, I=64, ld_a=128, live=P, ga=at(3), ld_ga=128) | change
    assert lib.megamoe_silu_mul_backward(*a.values(), P) == INVALID


@pytest.mark.parametrize("change", [
    dict(out=at(1)), dict(out=at(1, 3 * 64 * 2)), dict(x=at(3, 7 * 64 * 2)), dict(idx=at(3, 512))])
def test_rows(lib, change):
    a = dict(x=at(1), type=BF, T=4, d=64, ld_x=64, idx=at(2), rows=8, k=2, out=at(3), ld_out=64) | change
    assert lib.megamoe_gather_rows(*a.values(), P) == INVALID
    T, rows = 8, 4  # the other way round
    c = dict(y=a["x"], type=BF, rows=rows, ld=64, dst=a["idx"], w=P, T=T, k=2, d=64, out=a["out"], ld_out=64)
    assert lib.megamoe_combine_rows(*c.values(), P) == INVALID


@pytest.mark.parametrize("change", [
    dict(gy=at(1)), dict(gy=at(2, 128)), dict(gy=at(2), ld_gy=72), dict(gy=at(3)), dict(gy=at(4)),
    dict(gy=at(6)), dict(gw=at(1)), dict(gw=at(2)), dict(gw=at(3)), dict(gw=at(4, 4))])
def test_combine_backward(lib, change):
    a = dict(g=at(1), ld_g=64, y=at(2), type=BF, rows=8, ld_y=64, dst=at(3), w=at(4), T=4, k=2, d=64,
             gy=at(5), ld_gy=64, gw=at(6)) | change
    assert lib.megamoe_combine_rows_backward(*a.values(), P) == INVALID


@pytest.mark.parametrize("change", [dict(codes=at(1)), dict(scales=at(1, 64)), dict(scales=at(2, 16))])
def test_quantise(lib, change):
    a = dict(x=at(1), type=BF, rows=4, K=64, ld=64, codes=at(2), scales=at(3), status=P) | change
    assert lib.megamoe_quantize_int8(*a.values(), P) == INVALID


@pytest.mark.parametrize("T", [3, 12, 100])
@pytest.mark.parametrize("change", [
    dict(out=at(1)), dict(out=at(2)), dict(out=at(3)), dict(out=at(4)), dict(ws=at(1)), dict(ws=at(2)),
    dict(x=at(4)), dict(sw=at(4)), dict(type=I8, sx=at(5)), dict(type=I8, sx=at(4))])
def test_linear(lib, T, change):
    a = dict(x=at(1), type=BF, T=T, K=64, ld_x=64, sx=P, w=at(2), sw=at(3), N=72, epi=2, out=at(5), ld_out=72,
             ws=at(4), bytes=1 << 18) | change
    assert lib.megamoe_linear_int8(*a.values(), P) == INVALID
