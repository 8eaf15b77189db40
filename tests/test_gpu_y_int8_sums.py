"""The 8-bit linear's sums past 2^24, in each of its ways and on both sides of their limits:
an fp32 result is the integers' own sum, rounded once, times the two scales."""

import pytest
import torch

from nvfp4_block_scaled_topk_gb300 import megamoe

pytestmark = pytest.mark.gpu


def _large_codes(T, K, N, seed=0):
    """Codes of one sign and nearly the largest size, -128 among them."""
    g = torch.Generator().manual_seed(seed + T + K)
    q = torch.randint(97, 128, (T, K), generator=g, dtype=torch.int8)
    w = torch.randint(-128, -96, (N, K), generator=g, dtype=torch.int8)
    sx, sw = torch.rand(T, generator=g) + 0.5, torch.rand(N, generator=g) + 0.5
    return q.cuda(), w.cuda(), sx.cuda(), sw.cuda()


# up to 4 tokens, up to 16 (6016 is the longest row of 9 to 16, 12160 of 5 to 8)
@pytest.mark.parametrize("T,K", [(1, 4096), (2, 8192), (3, 1552), (4, 12304), (1, 49152), (5, 12160),
                                 (8, 7168), (8, 1040), (9, 6016), (16, 4112), (12, 6016)])
@pytest.mark.parametrize("N", [24, 2056])
def test_few_tokens_sum_exactly(cuda_lib, T, K, N):
    q, w, sx, sw = _large_codes(T, K, N)
    total = q.double() @ w.double().t()
    assert total.abs().min() > 2 ** 23 and total.abs().max() > 2 ** 24 - 2 ** 22
    want = total.float() * sx.unsqueeze(1) * sw  # the integers' sum, rounded once
    got, ws = megamoe.linear_int8(q, megamoe.Int8LinearWeights(N, K, w, sw), megamoe.EPI_F32, x_scales=sx)
    assert torch.equal(got, want) and int(ws[:4].view(torch.int32)) == 0


def test_a_token_has_one_result(cuda_lib):
    q, w, sx, sw = _large_codes(40, 6016, 520)
    weight = megamoe.Int8LinearWeights(520, 6016, w, sw)
    all_, _ = megamoe.linear_int8(q, weight, megamoe.EPI_F32, x_scales=sx)
    for T in [*range(1, 18), 33]:
        got, _ = megamoe.linear_int8(q[:T], weight, megamoe.EPI_F32, x_scales=sx[:T])
        assert torch.equal(got, all_[:T]), T


@pytest.mark.parametrize("T,K", [(5, 12176), (9, 6032), (16, 6032), (17, 4096), (40, 1040), (130, 2064),
                                 (300, 8192), (700, 1552)])
@pytest.mark.parametrize("N", [264, 5000])
def test_more_tokens_sum_exactly(cuda_lib, T, K, N):
    q, w, sx, sw = _large_codes(T, K, N)
    want = (q.double() @ w.double().t()).float() * sx.unsqueeze(1) * sw
    weight = megamoe.Int8LinearWeights(N, K, w, sw)
    got, ws = megamoe.linear_int8(q, weight, megamoe.EPI_F32, x_scales=sx)
    assert torch.equal(got, want) and int(ws[:4].view(torch.int32)) == 0
    again, _ = megamoe.linear_int8(q, weight, megamoe.EPI_F32, x_scales=sx, ws=ws)
    assert torch.equal(again, want)
    # bf16 results: one addition for each 16 of K, each cut by at most a unit of 2^-23 of the
    # sum so far (shares of a sum are shorter, with an addition each: no more than 16), two
    # scales, half a step
    got, _ = megamoe.linear_int8(q, weight, x_scales=sx, ws=ws)
    exact = (q.double() @ w.double().t()) * sx.double().unsqueeze(1) * sw.double()
    room = (K / 16 + 16 + 2) * 2.0 ** -23 * exact.abs()
    assert ((got.double() - exact).abs() <= room + (exact.abs() + room) * 2.0 ** -8).all()


def test_many_tiles_sum_exactly(cuda_lib):
    """More tiles than pairs of CTAs, parts of a sum that end inside a tile's steps."""
    q, w, sx, sw = _large_codes(1500, 2576, 3000)
    got, _ = megamoe.linear_int8(q, megamoe.Int8LinearWeights(3000, 2576, w, sw), megamoe.EPI_F32, x_scales=sx)
    assert torch.equal(got, (q.double() @ w.double().t()).float() * sx.unsqueeze(1) * sw)


def test_signs_that_cancel(cuda_lib):
    """Partial sums past 2^24 of which little is left."""
    q, w, sx, sw = _large_codes(40, 8192, 264)
    q[:, 4096:] = -q[:, :4096]
    q[:, ::7] //= 3
    for T in (3, 6, 40):
        got, _ = megamoe.linear_int8(q[:T], megamoe.Int8LinearWeights(264, 8192, w, sw), megamoe.EPI_F32,
                                     x_scales=sx[:T])
        want = (q[:T].double() @ w.double().t()).float() * sx[:T].unsqueeze(1) * sw
        assert torch.equal(got, want)


def test_rows_past_what_32_bits_hold(cuda_lib):
    """From 131072 terms on the sum is fp32's, each of its additions cut."""
    T, K, N = 20, 131072, 24
    q, w, sx, sw = _large_codes(T, K, N)
    got, _ = megamoe.linear_int8(q, megamoe.Int8LinearWeights(N, K, w, sw), megamoe.EPI_F32, x_scales=sx)
    want = (q.double() @ w.double().t()) * sx.double().unsqueeze(1) * sw.double()
    assert ((got.double() - want).abs() <= (K / 16 + 18) * 2.0 ** -23 * want.abs()).all()


@pytest.mark.parametrize("T", [4, 8, 16, 33, 200])
def test_the_largest_codes(cuda_lib, T):
    K, N = 4112, 264
    q = torch.full((T, K), -128, dtype=torch.int8, device="cuda")
    one = torch.ones(N, device="cuda")
    for b in (-128, 127, -127):
        w = torch.full((N, K), b, dtype=torch.int8, device="cuda")
        w[1, ::3] = 1
        got, _ = megamoe.linear_int8(q, megamoe.Int8LinearWeights(N, K, w, one), megamoe.EPI_F32,
                                     x_scales=torch.ones(T, device="cuda"))
        assert torch.equal(got, (q.double() @ w.double().t()).float())


@pytest.mark.parametrize("T", [8, 40, 700])
def test_waits_that_run_out(cuda_lib, T):
    """The word says so, and the next call is as if nothing had been."""
    q, w, sx, sw = _large_codes(T, 4112, 2056)
    weight = megamoe.Int8LinearWeights(2056, 4112, w, sw)
    want, ws = megamoe.linear_int8(q, weight, megamoe.EPI_F32, x_scales=sx)
    torch.cuda.synchronize()
    megamoe.set_wait_limit_ns(100)
    try:
        megamoe.linear_int8(q, weight, megamoe.EPI_F32, x_scales=sx, ws=ws)
        torch.cuda.synchronize()
        assert int(ws[:4].view(torch.int32)) == (megamoe.DEV_TIMEOUT if T > 16 else 0)
    finally:
        megamoe.set_wait_limit_ns(0)
    got, _ = megamoe.linear_int8(q, weight, megamoe.EPI_F32, x_scales=sx, ws=ws)
    assert torch.equal(got, want) and int(ws[:4].view(torch.int32)) == 0
