"""Offsets that give rows to two experts: the later one is left out and the status word
says so, whichever way the call takes; experts in any other order that share none."""

import pytest
import torch

from nvfp4_block_scaled_topk_gb300 import megamoe

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
U = 2.0 ** -23


def _run(starts, counts, rows, K, N, out_dtype=BF):
    """Status, result, gradients; rows that nothing wrote hold 7."""
    E = len(counts)
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn((rows, K), generator=g, device="cuda").to(BF)
    gr = torch.randn((rows, N), generator=g, device="cuda").to(BF)
    w = (torch.randn((E, N, K), generator=g, device="cuda") / 16).to(BF)
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = torch.tensor(counts).cumsum(0)
    poff = torch.tensor(starts + [rows], dtype=torch.int32).cuda()
    status = torch.zeros(3, dtype=torch.int32, device="cuda")
    y = torch.full((rows, N), 7.0, dtype=out_dtype, device="cuda")
    megamoe.grouped_linear(x, w, off.cuda(), poff, out_dtype=out_dtype, out=y, status=status[0:1])
    gx = torch.full((rows, K), 7.0, dtype=BF, device="cuda")
    megamoe.grouped_linear_backward(gr, x, w, off.cuda(), poff, need_w=False, grad_x=gx, status=status[1:2])
    _, gw = megamoe.grouped_linear_backward(gr, x, w, off.cuda(), poff, need_x=False, status=status[2:3])
    return status.tolist(), x, gr, w, y, gx, gw


def _check(values, owner, starts, counts):
    _, x, gr, w, y, gx, gw = values
    K, N = x.shape[1], gr.shape[1]

    def within(got, want, bound):
        eps = torch.finfo(got.dtype).eps
        assert ((got.double() - want).abs() <= bound + (want.abs() + bound) * eps / 2).all()

    for e in range(len(counts)):
        p, g, q = x[owner == e].double(), gr[owner == e].double(), w[e].double()
        within(y[owner == e], p @ q.t(), (K / 16 + 6) * U * (p.abs() @ q.abs().t()))
        within(gx[owner == e], g @ q, (N / 16 + 6) * U * (g.abs() @ q.abs()))
        within(gw[e], g.t() @ p, (len(p) / 16 + 6) * U * (g.abs().t() @ p.abs()))
        if not len(p):
            assert (gw[e] == 0).all()
    assert (y[owner < 0] == 7).all() and (gx[owner < 0] == 7).all()


SIZES = [(72, 136), (2056, 2120), (8200, 520)]  # a sum by one pair of CTAs, by two, by more


@pytest.mark.parametrize("K,N", SIZES)
@pytest.mark.parametrize("out_dtype", [BF, torch.float32])
@pytest.mark.parametrize("starts,counts,left", [
    ([0, 4, 20], [8, 8, 6], [1]),            # the second begins inside the first
    ([0, 0, 0], [10, 10, 10], [1, 2]),       # all the same
    ([10, 0, 12], [6, 12, 0], [1]),          # ... or ends in it; none of no rows
    ([0, 8, 3], [8, 8, 2], [2]),             # one inside another
    ([0, 5, 10], [30, 5, 16], [1, 2])])
def test_shared_rows(cuda_lib, K, N, out_dtype, starts, counts, left):
    rows = 32
    values = _run(starts, counts, rows, K, N, out_dtype)
    assert values[0] == [megamoe.DEV_BAD_OFFSETS] * 3
    owner = torch.full((rows,), -1, device="cuda")
    for e, (s, c) in enumerate(zip(starts, counts)):
        if e not in left:
            owner[s:s + c] = e
    _check(values, owner, starts, counts)


@pytest.mark.parametrize("K,N", SIZES)
def test_any_order(cuda_lib, K, N):
    starts, counts, rows = [20, 0, 9, 9, 31], [11, 8, 0, 10, 1], 32
    values = _run(starts, counts, rows, K, N)
    assert values[0] == [0] * 3
    owner = torch.full((rows,), -1, device="cuda")
    for e, (s, c) in enumerate(zip(starts, counts)):
        owner[s:s + c] = e
    _check(values, owner, starts, counts)


def test_many_experts(cuda_lib):
    """More experts than threads; every third one lies in the row of the one before."""
    E = 1000
    starts = [e - e // 3 if e % 3 < 2 else e - e // 3 - 1 for e in range(E)]
    rows = max(starts) + 1
    values = _run(starts, [1] * E, rows, 64, 72)
    assert values[0] == [megamoe.DEV_BAD_OFFSETS] * 3
    owner = torch.full((rows,), -1, device="cuda")
    for e, s in enumerate(starts):
        if owner[s] < 0:
            owner[s] = e
    assert (owner >= 0).all()
    x, gr, w, y, gx, gw = values[1:]
    wo = w[owner].double()
    want, most = (torch.einsum("rk,rnk->rn", a, b) for a, b in ((x.double(), wo), (x.double().abs(), wo.abs())))
    bound = 6 * U * most
    assert ((y.double() - want).abs() <= bound + (want.abs() + bound) * 2.0 ** -8).all()
    lives = torch.zeros(E, dtype=torch.bool, device="cuda")
    lives[owner] = True
    assert (gw[~lives] == 0).all()
    want = gr.double()[:, :, None] * x.double()[:, None, :]
    assert torch.equal(gw[owner].double(), want)  # one row: products of two are exact
