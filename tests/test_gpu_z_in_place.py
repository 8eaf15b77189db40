"""Results in place where that is allowed, between the rows of what a call reads, and the
binding's refusal of the rest."""

import pytest
import torch

from nvfp4_block_scaled_topk_gb300 import megamoe

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _normal(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(BF)


@pytest.mark.parametrize("rows,I", [(1, 8), (37, 264), (3000, 1024)])
def test_activation(cuda_lib, rows, I):
    a, grad = _normal(rows, 2 * I), _normal(rows, I, seed=1)
    want, want_grad = megamoe.silu_mul(a), megamoe.silu_mul_backward(grad, a)
    for columns in (slice(0, I), slice(I, 2 * I)):
        b = a.clone()
        out = megamoe.silu_mul(b, out=b[:, columns])
        assert torch.equal(out, want)
        other = slice(I, 2 * I) if columns.start == 0 else slice(0, I)
        assert torch.equal(b[:, other], a[:, other])
        wide = torch.zeros_like(a)
        wide[:, columns] = grad
        assert torch.equal(megamoe.silu_mul_backward(wide[:, columns], a, grad_a=wide), want_grad)
    b = a.clone()
    assert torch.equal(megamoe.silu_mul_backward(grad, b, grad_a=b), want_grad)


@pytest.mark.parametrize("T,k,d", [(1, 1, 8), (300, 6, 1032), (9, 16, 72)])
def test_gradient_of_the_sums(cuda_lib, T, k, d):
    y, grad = _normal(T * k, d), _normal(T, d, seed=1)
    dst = torch.randperm(T * k, device="cuda").int().view(T, k)
    w = torch.rand((T, k), device="cuda")
    want = megamoe.combine_rows_backward(grad, y, dst, w)
    got = megamoe.combine_rows_backward(grad, y, dst, w, grad_y=y)
    assert got[0] is y and torch.equal(y, want[0]) and torch.equal(got[1], want[1])


def test_between_the_rows_of_the_operands(cuda_lib):
    K, N, R = 72, 136, 50
    wide = _normal(R, K + N)
    w = _normal(2, N, K, seed=1)
    off = torch.tensor([0, 20, R], dtype=torch.int32, device="cuda")
    x, grad = wide[:, :K].contiguous(), wide[:, K:].contiguous()
    want = megamoe.grouped_linear(x, w, off)
    gx, gw = megamoe.grouped_linear_backward(grad, x, w, off)
    b = wide.clone()
    assert torch.equal(megamoe.grouped_linear(b[:, :K], w, off, out=b[:, K:]), want)
    assert torch.equal(b[:, :K], x)
    b = wide.clone()  # x is not read where grad_w is not asked for
    assert torch.equal(megamoe.grouped_linear_backward(b[:, K:], b[:, :K], w, off, need_w=False,
                                                       grad_x=b[:, :K])[0], gx)
    weight = megamoe.Int8LinearWeights.quantize(_normal(N, 64, seed=2))
    for T in (3, 12, 50):
        want = megamoe.linear_int8(wide[:T, :64], weight)[0]
        b = wide.clone()
        assert torch.equal(megamoe.linear_int8(b[:T, :64], weight, out=b[:T, K:])[0], want)


def test_refusals(cuda_lib):
    x, y, w = _normal(6, 64), _normal(6, 64), _normal(2, 64, 64)
    off = torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda")
    weight = megamoe.Int8LinearWeights.quantize(_normal(64, 64))
    dst = torch.arange(6, dtype=torch.int32, device="cuda").view(6, 1)
    for call in (lambda: megamoe.grouped_linear(x, w, off, out=x),
                 lambda: megamoe.grouped_linear_backward(x, y, w, off, grad_x=x),
                 lambda: megamoe.grouped_linear_backward(y, x, w, off, grad_x=x),
                 lambda: megamoe.grouped_linear_backward(y, x, w, off, grad_x=w[1, :6]),
                 lambda: megamoe.silu_mul(x, out=x[:, 16:48]),
                 lambda: megamoe.silu_mul_backward(x[:3].view(6, 32), y, grad_a=x),
                 lambda: megamoe.gather_rows(x, dst.view(6), 1, out=x),
                 lambda: megamoe.combine_rows(x, dst, out=x),
                 lambda: megamoe.combine_rows_backward(x, y, dst, grad_y=x),
                 lambda: megamoe.linear_int8(x, weight, out=x)):
        with pytest.raises(megamoe.MegaMoEError):
            call()
