"""The 8-bit linear's scales where the sum times one of them alone leaves fp32's range."""

import pytest
import torch

from nvfp4_block_scaled_topk_gb300 import megamoe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 4, 8, 16, 40, 400])
@pytest.mark.parametrize("x_scale,w_scale", [(2.0 ** 120, 2.0 ** -40), (2.0 ** 100, 2.0 ** -100),
                                             (2.0 ** 66, 2.0 ** 20), (2.0 ** -120, 2.0 ** 90),
                                             (2.0 ** -140, 2.0 ** 127), (2.0 ** 40, 2.0 ** 60)])
def test_scales_far_apart(cuda_lib, T, x_scale, w_scale):
    """The sum times either scale alone may leave fp32's range; the result does not."""
    g = torch.Generator().manual_seed(T)
    q = torch.randint(-20, 21, (T, 2064), generator=g, dtype=torch.int8).cuda()
    w = torch.randint(-20, 21, (264, 2064), generator=g, dtype=torch.int8).cuda()
    sx = (torch.rand(T, generator=g) + 0.5).mul(x_scale).cuda()
    sw = (torch.rand(264, generator=g) + 0.5).mul(w_scale).cuda()
    weight = megamoe.Int8LinearWeights(264, 2064, w, sw)
    total = q.double() @ w.double().t()  # below 2^24
    want = total * sx.double().unsqueeze(1) * sw.double()
    assert want.abs().max() < 3e38
    for epi, half in ((megamoe.EPI_F32, 0.0), (megamoe.EPI_BF16, 2.0 ** -8)):
        got, ws = megamoe.linear_int8(q, weight, epi, x_scales=sx)
        room = 2 * 2.0 ** -24 * want.abs() + 2.0 ** -149  # two products
        assert ((got.double() - want).abs() <= room + half * (want.abs() + room) + half * 2.0 ** -126).all()
        assert int(ws[:4].view(torch.int32)) == 0


@pytest.mark.parametrize("T", [4, 12, 300])
def test_a_loud_token_among_others(cuda_lib, T):
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, 1040), generator=g)
    loud = torch.arange(T) % 7 == 2
    x[loud] *= 2.0 ** 118
    x = x.cuda()
    weight = megamoe.Int8LinearWeights.quantize((torch.randn((520, 1040), generator=g) * 2.0 ** -30).cuda())
    codes, scales = megamoe.quantize_int8(x)
    want = (codes.double() @ weight.codes.double().t()) * scales.double().unsqueeze(1) * weight.scales.double()
    got, ws = megamoe.linear_int8(x, weight, megamoe.EPI_F32)
    assert ((got.double() - want).abs() <= 2 * 2.0 ** -24 * want.abs()).all()
    assert int(ws[:4].view(torch.int32)) == 0 and got[loud].abs().max() > 2.0 ** 88
    quiet, _ = megamoe.linear_int8(x[~loud], weight, megamoe.EPI_F32)
    assert torch.equal(quiet, got[~loud])
