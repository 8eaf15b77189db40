"""Quantisation to 8-bit integers and the integer linear against exact arithmetic.

Integers and scales are exact.  While sum |q_x q_w| stays below 2^24 the sum of
products is exact, and an fp32 result is that sum times the two scales, each
product rounded: the same bits.  Past that each of the K / 16 additions is off by
at most one unit of 2^-23 of what has been added up."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from nvfp4_block_scaled_topk_gb300 import megamoe

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


def strided(t, extra=16):
    return torch.cat([t, torch.full((t.shape[0], extra), 9, dtype=t.dtype, device=t.device)],
                     1)[:, :t.shape[1]]


def exact_codes(x):
    """Integers and fp32 scales of rows, decided by whole numbers."""
    x = x.double().cpu().numpy()
    codes = np.zeros(x.shape, np.int8)
    scales = np.zeros(len(x), np.float32)
    for t, row in enumerate(x):
        amax = np.abs(row).max() if row.size else 0.0
        if amax == 0:
            continue
        scales[t] = np.float32(amax) / np.float32(127)
        near = row * 127 / amax
        q = np.rint(near)
        for i in np.flatnonzero(np.abs(np.abs(near - np.floor(near)) - 0.5) < 1e-9):
            q[i] = round(Fraction(row[i]) * 127 / Fraction(amax))  # ties to even
        codes[t] = q
    return codes, scales


@pytest.mark.parametrize("rows,K", [(1, 16), (3, 64), (70, 1552), (5, 8192), (2, 8208), (2, 24576)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_quantise_exact(cuda_lib, rows, K, dtype):
    g = torch.Generator().manual_seed(rows + K)
    x = (torch.randn(rows, K, generator=g) * torch.exp2(torch.randint(-9, 6, (rows, 1), generator=g).float()))
    x = x.to(dtype)
    want = exact_codes(x)
    for xs in (x.cuda(), strided(x.cuda())):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        codes, scales = megamoe.quantize_int8(xs, status)
        assert np.array_equal(codes.cpu().numpy(), want[0])
        assert np.array_equal(scales.cpu().numpy(), want[1]) and int(status) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_quantise_ties_and_ends(cuda_lib, dtype):
    f = torch.finfo(dtype)
    big = torch.arange(-127, 128).repeat(2)[:256].double() / 2  # ties at every half
    rows = [big / 63.5 * 127, torch.zeros(256).double(), torch.full((256,), f.max).double(),
            torch.full((256,), -f.smallest_normal).double(),
            torch.arange(256).double() * f.smallest_normal * f.eps,  # subnormals
            torch.linspace(-1, 1, 256).double() * f.max]
    rows[0][0] = 127
    rows[0][1:] = torch.arange(255).double() / 2 - 63.5
    x = torch.stack(rows).to(dtype)
    codes, scales = megamoe.quantize_int8(x.cuda())
    want = exact_codes(x)
    assert np.array_equal(codes.cpu().numpy(), want[0])
    assert np.array_equal(scales.cpu().numpy(), want[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_quantise_rows_of_any_size(cuda_lib, dtype):
    """Rows whose largest magnitude has every mantissa of few bits (which make halves
    common) and every exponent that the type holds, elements of few bits among them."""
    f = torch.finfo(dtype)
    g = torch.Generator().manual_seed(8)
    low, high = int(np.log2(f.smallest_normal * f.eps)), int(np.floor(np.log2(f.max)))
    rows = []
    for e in range(low, high + 1, 3 if dtype == torch.float16 else 9):
        for mantissa in (128, 192, 160, 224, 129, 255):
            x = torch.randint(-mantissa, mantissa + 1, (256,), generator=g).double()
            x[:64] = (torch.rand(64, generator=g, dtype=torch.float64) * 2 - 1) * mantissa
            x[100] = mantissa
            rows.append(torch.ldexp(x, torch.tensor(e - 7)))
    x = torch.stack(rows).clamp(-f.max, f.max).to(dtype)
    codes, scales = megamoe.quantize_int8(x.cuda())
    want = exact_codes(x)
    assert np.array_equal(codes.cpu().numpy(), want[0])
    assert np.array_equal(scales.cpu().numpy(), want[1])
    w = megamoe.Int8LinearWeights.quantize(torch.eye(256, device="cuda"))
    for T in (1, 4, 12):  # the tokens' integers in a product with 127 at their own place
        out, _ = megamoe.linear_int8(x[5:5 + T].cuda(), w, megamoe.EPI_F32)
        with np.errstate(all="ignore"):
            prod = want[0][5:5 + T].astype(np.float32) * 127 * want[1][5:5 + T, None]
            assert np.array_equal(out.cpu().numpy(), prod * w.scales.cpu().numpy())


def test_quantise_nonfinite(cuda_lib):
    x = torch.randn(4, 64)
    x[1, 5], x[2, 63] = float("inf"), float("nan")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    codes, scales = megamoe.quantize_int8(x.cuda(), status)
    assert int(status) == megamoe.DEV_NONFINITE
    assert torch.isnan(scales[1:3]).all() and (codes[1:3] == 0).all()
    want = exact_codes(x[[0, 3]])
    assert np.array_equal(codes.cpu().numpy()[[0, 3]], want[0])
    w = megamoe.Int8LinearWeights.quantize(torch.randn(24, 64, device="cuda"))
    for T in (4, 40):
        out, ws = megamoe.linear_int8(x.repeat(T // 4, 1).cuda(), w)
        assert int(ws[:4].view(torch.int32)) == megamoe.DEV_NONFINITE
        bad = torch.isnan(out).all(1).view(-1, 4)
        assert bad[:, 1:3].all() and torch.isfinite(out.view(-1, 4, 24)[:, [0, 3]]).all()
        out, ws = megamoe.linear_int8(x[:1].repeat(T, 1).cuda(), w, ws=ws)  # the word is cleared
        assert int(ws[:4].view(torch.int32)) == 0 and torch.isfinite(out).all()


SHAPES = [(1, 64, 64), (1, 16, 8), (3, 144, 264), (8, 1536, 2048), (9, 48, 40), (17, 7168, 520),
          (40, 128, 1000), (130, 400, 264), (200, 272, 256), (257, 656, 72), (300, 1552, 2056),
          (513, 128, 24), (5, 8192, 5000)]


def _case(T, K, N, seed=0, most=127):
    g = torch.Generator().manual_seed(seed + T + K)
    q = torch.randint(-most, most + 1, (T, K), generator=g, dtype=torch.int8)
    w = torch.randint(-most, most + 1, (N, K), generator=g, dtype=torch.int8)
    sx = torch.rand(T, generator=g) + 0.5
    sw = torch.rand(N, generator=g) + 0.5
    return q.cuda(), w.cuda(), sx.cuda(), sw.cuda()


@pytest.mark.parametrize("T,K,N", SHAPES)
def test_linear_codes(cuda_lib, T, K, N):
    q, w, sx, sw = _case(T, K, N, most=40)
    weight = megamoe.Int8LinearWeights(N, K, w, sw)
    total = q.double().abs() @ w.double().abs().t()
    assert total.max() < 2 ** 24
    acc = (q.double() @ w.double().t()).float()
    want = acc * sx.unsqueeze(1) * sw
    wide = torch.full((T, N + 8), 7.0, device="cuda")
    got, ws = megamoe.linear_int8(strided(q), weight, megamoe.EPI_F32, x_scales=sx, out=wide[:, :N])
    assert torch.equal(got, want) and (wide[:, N:] == 7).all()
    assert int(ws[:4].view(torch.int32)) == 0
    got, _ = megamoe.linear_int8(q, weight, x_scales=sx, ws=ws)
    assert got.dtype == torch.bfloat16 and torch.equal(got, want.bfloat16())


@pytest.mark.parametrize("T,K,N", [(1, 8192, 264), (33, 8192, 264), (8, 4096, 8)])
def test_linear_extremes(cuda_lib, T, K, N):
    """Integers of the largest size, -128 among them, all of one sign: sums past 2^24."""
    for a, b in ((127, 127), (-128, -128), (-128, 127)):
        q = torch.full((T, K), a, dtype=torch.int8, device="cuda")
        w = torch.full((N, K), b, dtype=torch.int8, device="cuda")
        w[1, ::2] = 0
        one = torch.ones(N, device="cuda")
        got, _ = megamoe.linear_int8(q, megamoe.Int8LinearWeights(N, K, w, one), megamoe.EPI_F32,
                                     x_scales=torch.ones(T, device="cuda"))
        want = q.double() @ w.double().t()
        assert ((got.double() - want).abs() <= (K / 16 + 2) * U * want.abs()).all()


@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_linear(cuda_lib, T, K, N, dtype):
    g = torch.Generator().manual_seed(T + N)
    x = (torch.randn(T, K, generator=g) * 0.1).to(dtype).cuda()
    master = (torch.randn(N, K, generator=g) * 0.05).cuda()
    weight = megamoe.Int8LinearWeights.quantize(master)
    codes, scales = megamoe.quantize_int8(x)
    p, q = codes.double(), weight.codes.double()
    s = scales.double().unsqueeze(1) * weight.scales.double()
    want = (p @ q.t()) * s
    bound = ((K / 16 + 2) * U * (p.abs() @ q.abs().t()) * s) + 2 * 2.0 ** -24 * want.abs()
    for epi, half in ((megamoe.EPI_F32, 0.0), (megamoe.EPI_BF16, 2.0 ** -8)):
        got, ws = megamoe.linear_int8(strided(x), weight, epi)
        assert ((got.double() - want).abs() <= bound + half * (want.abs() + bound)).all()
        assert int(ws[:4].view(torch.int32)) == 0
        # the same bits from the codes, and again
        same, _ = megamoe.linear_int8(codes, weight, epi, x_scales=scales)
        assert torch.equal(same, got)
        assert torch.equal(megamoe.linear_int8(x, weight, epi, ws=ws)[0], got)


def test_linear_no_tokens(cuda_lib):
    w = megamoe.Int8LinearWeights.quantize(torch.randn(24, 64, device="cuda"))
    out, ws = megamoe.linear_int8(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), w)
    assert out.shape == (0, 24)
    assert int(ws[:4].view(torch.int32)) == 0
