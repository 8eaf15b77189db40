"""Argument checks and sizes of the 16-bit experts' operators and the 8-bit integer
linear, without a GPU: every refusal comes before any device work."""

import ctypes

import pytest
import torch

import __graft_entry__
from nvfp4_block_scaled_topk_gb300 import megamoe

P = None
F = ctypes.c_void_p(256)  # an aligned address that is never touched
ODD = ctypes.c_void_p(258)
INVALID, SHAPE, SMALL = 1, 2, 3
BF, F32, F16, I8 = 0, 1, 2, 3
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return megamoe.load()


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), INVALID), (dict(E=0), INVALID), (dict(N=0), INVALID), (dict(K=-8), INVALID),
    (dict(type=F32), INVALID), (dict(type=I8), INVALID), (dict(out_type=F16), INVALID),
    (dict(out_type=9), INVALID), (dict(x=P), INVALID), (dict(w=P), INVALID), (dict(out=P), INVALID),
    (dict(off=P), INVALID), (dict(ld_x=56), INVALID), (dict(ld_out=64), INVALID),
    (dict(E=1025), SHAPE), (dict(rows=1 << 30, E=1), SHAPE), (dict(K=60), SHAPE), (dict(N=68), SHAPE),
    (dict(x=ODD), SHAPE), (dict(w=ODD), SHAPE), (dict(out=ODD), SHAPE), (dict(off=ODD), SHAPE),
    (dict(poff=ODD), SHAPE), (dict(status=ODD), SHAPE), (dict(ld_x=66), SHAPE),
    (dict(ld_out=74), SHAPE), (dict(ld_out=1 << 36), SHAPE),
    (dict(out_type=F32, ld_out=74), SHAPE), (dict(K=1 << 30, ld_x=1 << 30), SHAPE),
    (dict(N=1 << 29, K=1 << 12, ld_x=1 << 12, ld_out=1 << 29), SHAPE),
    (dict(rows=1 << 30, E=1024), SHAPE)])
def test_grouped_refusals(lib, change, code):
    a = dict(x=F, type=BF, rows=40, ld_x=64, w=F, E=4, N=72, K=64, off=F, poff=P, out_type=BF, out=F,
             ld_out=72, status=P) | change
    assert lib.megamoe_grouped_linear(*a.values(), P) == code


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), INVALID), (dict(type=F32), INVALID), (dict(g=P), INVALID), (dict(x=P), INVALID),
    (dict(w=P), INVALID), (dict(off=P), INVALID), (dict(ld_g=64), INVALID), (dict(ld_x=56), INVALID),
    (dict(ld_gx=56), INVALID), (dict(w_type=F16), INVALID), (dict(w_type=I8), INVALID),
    (dict(E=1025), SHAPE), (dict(N=68, ld_g=72), SHAPE), (dict(K=60), SHAPE), (dict(g=ODD), SHAPE),
    (dict(x=ODD), SHAPE), (dict(w=ODD), SHAPE), (dict(gx=ODD), SHAPE), (dict(gw=ODD), SHAPE),
    (dict(ld_g=76), SHAPE), (dict(ld_gx=66), SHAPE), (dict(status=ODD), SHAPE)])
def test_grouped_backward_refusals(lib, change, code):
    a = dict(g=F, ld_g=72, x=F, ld_x=64, w=F, type=F16, rows=40, E=4, N=72, K=64, off=F, poff=P, gx=F,
             ld_gx=64, w_type=F32, gw=F, status=P) | ({"w_type": BF} if change == dict(w_type=F16) else change)
    assert lib.megamoe_grouped_linear_backward(*a.values(), P) == code


@pytest.mark.parametrize("change,code", [
    (dict(type=F32), INVALID), (dict(rows=-1), INVALID), (dict(I=0), INVALID), (dict(a=P), INVALID),
    (dict(out=P), INVALID), (dict(ld_a=120), INVALID), (dict(ld_out=56), INVALID), (dict(I=60), SHAPE),
    (dict(a=ODD), SHAPE), (dict(out=ODD), SHAPE), (dict(live=ODD), SHAPE), (dict(ld_a=132), SHAPE),
    (dict(rows=BIG), SHAPE)])
def test_silu_refusals(lib, change, code):
    a = dict(a=F, type=BF, rows=4, I=64, ld_a=128, live=P, out=F, ld_out=64) | change
    assert lib.megamoe_silu_mul(*a.values(), P) == code
    b = dict(g=F, ld_g=64, a=F, type=BF, rows=4, I=64, ld_a=128, live=P, ga=F, ld_ga=128)
    b |= {{"out": "g", "ld_out": "ld_g"}.get(k, k): v for k, v in change.items()}
    assert lib.megamoe_silu_mul_backward(*b.values(), P) == code
    assert lib.megamoe_silu_mul_backward(*(b | dict(ga=P)).values(), P) != 0


@pytest.mark.parametrize("change,code", [
    (dict(type=F32), INVALID), (dict(T=-1), INVALID), (dict(rows=-1), INVALID), (dict(k=0), INVALID),
    (dict(d=0), INVALID), (dict(x=P), INVALID), (dict(idx=P), INVALID), (dict(out=P), INVALID),
    (dict(ld_x=56), INVALID), (dict(ld_out=56), INVALID), (dict(d=60), SHAPE), (dict(k=17), SHAPE),
    (dict(x=ODD), SHAPE), (dict(idx=ODD), SHAPE), (dict(out=ODD), SHAPE), (dict(rows=BIG), SHAPE),
    (dict(T=BIG), SHAPE)])
def test_rows_refusals(lib, change, code):
    a = dict(x=F, type=BF, T=4, d=64, ld_x=64, idx=F, rows=8, k=2, out=F, ld_out=64) | change
    assert lib.megamoe_gather_rows(*a.values(), P) == code
    c = dict(y=a["x"], type=a["type"], rows=a["rows"], ld=a["ld_x"], dst=a["idx"], w=P, T=a["T"],
             k=a["k"], d=a["d"], out=a["out"], ld_out=a["ld_out"])
    assert lib.megamoe_combine_rows(*c.values(), P) == code
    b = dict(g=a["x"], ld_g=a["ld_x"], y=F, type=a["type"], rows=a["rows"], ld_y=64, dst=a["idx"], w=P,
             T=a["T"], k=a["k"], d=a["d"], gy=a["out"], ld_gy=a["ld_out"], gw=P)
    assert lib.megamoe_combine_rows_backward(*b.values(), P) == code


@pytest.mark.parametrize("change,code", [
    (dict(w=ODD), SHAPE), (dict(gw=ODD), SHAPE), (dict(y=P), INVALID), (dict(ld_y=56), INVALID),
    (dict(y=ODD), SHAPE), (dict(ld_y=66), SHAPE)])
def test_combine_backward_refusals(lib, change, code):
    a = dict(g=F, ld_g=64, y=F, type=BF, rows=8, ld_y=64, dst=F, w=F, T=4, k=2, d=64, gy=F, ld_gy=64,
             gw=F) | change
    assert lib.megamoe_combine_rows_backward(*a.values(), P) == code


@pytest.mark.parametrize("change,code", [
    (dict(type=I8), INVALID), (dict(type=7), INVALID), (dict(rows=-1), INVALID), (dict(K=0), INVALID),
    (dict(ld=48), INVALID), (dict(x=P), INVALID), (dict(codes=P), INVALID), (dict(scales=P), INVALID),
    (dict(K=56), SHAPE), (dict(ld=68), SHAPE), (dict(x=ODD), SHAPE), (dict(codes=ODD), SHAPE),
    (dict(scales=ODD), SHAPE), (dict(status=ODD), SHAPE), (dict(rows=BIG), SHAPE)])
def test_quantise_refusals(lib, change, code):
    a = dict(x=F, type=BF, rows=4, K=64, ld=64, codes=F, scales=F, status=P) | change
    assert lib.megamoe_quantize_int8(*a.values(), P) == code


@pytest.mark.parametrize("T", [3, 12, 100])  # each of the three ways
@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(K=0), INVALID), (dict(N=0), INVALID), (dict(type=9), INVALID),
    (dict(ld_x=48), INVALID), (dict(ld_out=64), INVALID), (dict(x=P), INVALID), (dict(w=P), INVALID),
    (dict(sw=P), INVALID), (dict(out=P), INVALID), (dict(ws=P), INVALID), (dict(epi=1), INVALID),
    (dict(epi=3), INVALID), (dict(sx=F), INVALID), (dict(type=I8), INVALID), (dict(K=56), SHAPE),
    (dict(N=68), SHAPE), (dict(ld_x=68), SHAPE), (dict(ld_out=74), SHAPE), (dict(x=ODD), SHAPE),
    (dict(w=ODD), SHAPE), (dict(sw=ODD), SHAPE), (dict(out=ODD), SHAPE), (dict(ws=ODD), SHAPE),
    (dict(type=I8, sx=ODD), SHAPE), (dict(type=I8, sx=F, ld_x=72), SHAPE),
    (dict(T=1 << 30), SHAPE), (dict(K=1 << 30, ld_x=1 << 30), SHAPE), (dict(bytes=255), SMALL)])
def test_linear_refusals(lib, T, change, code):
    a = dict(x=F, type=BF, T=T, K=64, ld_x=64, sx=P, w=F, sw=F, N=72, epi=2, out=F, ld_out=72, ws=F,
             bytes=1 << 30) | change
    if change.get("type") == I8 and "sx" not in change:
        a["sx"] = P  # codes without scales
    # an odd pair of types: rows of 8-bit codes on 16-byte boundaries
    assert lib.megamoe_linear_int8(*a.values(), P) == code


def test_workspace_sizes(lib):
    size = lib.megamoe_linear_int8_workspace_size
    assert size(-1, 64, 64) == 0 and size(4, 0, 64) == 0 and size(4, 56, 64) == 0
    assert size(4, 64, 60) == 0 and size(1 << 30, 64, 64) == 0
    assert size(0, 64, 64) >= 256 and size(1, 1536, 24576) == 256
    few, pair = size(12, 7168, 2048), size(100, 7168, 2048)
    assert few >= 256 + 12 * 4 + 12 * 7168
    # shares of a sum: fp32 [split][T][N] behind the integers
    assert pair >= 256 + 100 * 4 + 2 * 100 * 7168 + 2 * 4 * 100 * 2048
    assert size(8192, 7168, 2048) < 256 + 8192 * 4 + 2 * 8192 * 7168 + 1024
    for bytes_, T in ((few, 12), (pair, 100)):
        assert lib.megamoe_linear_int8(F, BF, T, 7168, 7168, P, F, F, 2048, 2, F, 2048, F, bytes_ - 1,
                                       P) == SMALL


def test_binding_refuses_host_tensors(lib):
    x, w = torch.zeros(4, 64).bfloat16(), torch.zeros(2, 64, 64).bfloat16()
    off = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: megamoe.grouped_linear(x, w, off),
                 lambda: megamoe.grouped_linear_backward(x, x, w, off),
                 lambda: megamoe.silu_mul(x), lambda: megamoe.silu_mul_backward(x, x),
                 lambda: megamoe.gather_rows(x, off, 2), lambda: megamoe.combine_rows(x, off.view(3, 1)),
                 lambda: megamoe.combine_rows_backward(x, x, off.view(3, 1)),
                 lambda: megamoe.quantize_int8(x),
                 lambda: megamoe.Int8LinearWeights(4, 64, x.to(torch.int8), torch.zeros(4))):
        with pytest.raises(TypeError):
            call()
