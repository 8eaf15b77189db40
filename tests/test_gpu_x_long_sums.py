"""Products grouped by expert in 16 bits whose sums have a million terms, all of one
sign, so that what the tensor cores' sums drop adds up.

Parts of 1024 terms: 64 additions, each off by at most one unit of 2^-23 of what has
been added up; the parts by fp32 additions, each off by 2^-24 at most.  A result so is
within 66 2^-23 + P 2^-24 of the sum (P parts; pairs that share a sum add three more),
and half a step of its type."""

import pytest
import torch

from nvfp4_block_scaled_topk_gb300 import megamoe

pytestmark = pytest.mark.gpu

LONG = 1 << 20


def _positive(g, shape, top):
    """[top / 2, top]"""
    return ((torch.rand(shape, generator=g, device="cuda") + 1) * (top / 2)).half()


def _check(got, want, terms):
    room = (66 * 2.0 ** -23 + (terms / 1024 + 4) * 2.0 ** -24) * want.abs()
    err = (got.double() - want).abs()
    bound = room + (want.abs() + room) * torch.finfo(got.dtype).eps / 2
    assert (err <= bound).all(), (err / want.abs()).max()


def test_gradient_of_weights(cuda_lib):
    g = torch.Generator(device="cuda").manual_seed(1)
    R, K, N = LONG + 40, 24, 40  # the second expert's rows end inside a tile
    off = torch.tensor([0, 33, R], dtype=torch.int32, device="cuda")
    x, gr = _positive(g, (R, K), 1.0), _positive(g, (R, N), 2.0 ** -6)
    w = _positive(g, (2, N, K), 1.0)
    gx, gw = megamoe.grouped_linear_backward(gr, x, w, off, grad_w_dtype=torch.float16)
    _check(gw[0], gr[:33].double().t() @ x[:33].double(), 33)
    _check(gw[1], gr[33:].double().t() @ x[33:].double(), LONG)
    _check(gx[-64:], gr[-64:].double() @ w[1].double(), N)


@pytest.mark.parametrize("E,terms", [(1, LONG), (36, LONG // 4)])  # shared sums, and not
def test_forward_and_gradient_of_rows(cuda_lib, E, terms):
    g = torch.Generator(device="cuda").manual_seed(E)
    rows = 2 * E
    off = torch.arange(0, rows + 1, 2, dtype=torch.int32, device="cuda")
    x = _positive(g, (rows, terms), 1.0)
    w = _positive(g, (E, 8, terms), 2.0 ** -6)
    want = torch.cat([x[2 * e:2 * e + 2].double() @ w[e].double().t() for e in range(E)])
    _check(megamoe.grouped_linear(x, w, off), want, terms)
    wt = w.transpose(1, 2).contiguous()  # [E, terms, 8]: grad_x sums over them
    y = torch.zeros((rows, 8), dtype=torch.float16, device="cuda")
    gx, _ = megamoe.grouped_linear_backward(x, y, wt, off, need_w=False)
    _check(gx, want, terms)
