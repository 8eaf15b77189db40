"""Tensors that the MXFP4 entry points of the binding refuse before anything is
launched: on the host, of another type, strided, too small (a workspace may be of any type)."""

import pytest
import torch

from nvfp4_block_scaled_topk_gb300 import megamoe

pytestmark = pytest.mark.gpu

T, K, N = 100, 256, 64


def _x(rows=T, cols=K):
    return torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")


def _bad_workspaces(size):
    cuda = torch.zeros(2 * size, dtype=torch.uint8, device="cuda")
    return [torch.zeros(size, dtype=torch.uint8), cuda[::2], cuda[:1].expand(size)]


def test_workspaces(cuda_lib):
    w = megamoe.MxLinearWeights.quantize(_x(N, K))
    out, good = megamoe.linear_mxfp4(_x(), w)
    for ws in _bad_workspaces(good.numel()):
        with pytest.raises(TypeError):
            megamoe.linear_mxfp4(_x(), w, ws=ws)
    with pytest.raises(megamoe.MegaMoEError):
        megamoe.linear_mxfp4(_x(), w, ws=good[:-1])
    words = torch.zeros(good.numel() // 4 + 1, dtype=torch.int32, device="cuda")
    for ws in (good, words):
        assert torch.equal(megamoe.linear_mxfp4(_x(), w, ws=ws)[0], out)
    args = (_x(T, N), _x(), _x(N, K))
    gx, gw, good = megamoe.linear_mxfp4_backward(*args)
    for ws in _bad_workspaces(good.numel()):
        with pytest.raises(TypeError):
            megamoe.linear_mxfp4_backward(*args, ws=ws)
    with pytest.raises(megamoe.MegaMoEError):
        megamoe.linear_mxfp4_backward(*args, ws=good[:-1])
    again = megamoe.linear_mxfp4_backward(*args, ws=good)
    assert torch.equal(again[0], gx) and torch.equal(again[1], gw)


def test_weights(cuda_lib):
    w = megamoe.MxLinearWeights.quantize(_x(N, K))
    for codes, scales in ((w.codes.cpu(), w.scales), (w.codes, w.scales.cpu()),
                          (w.codes.float(), w.scales), (w.codes.t(), w.scales)):
        with pytest.raises(TypeError):
            megamoe.MxLinearWeights(N, K, codes, scales)
    for n, k in ((N + 32, K), (N, K + 32)):
        with pytest.raises(ValueError):
            megamoe.MxLinearWeights(n, k, w.codes, w.scales)
    E, d, I = 2, 256, 256
    raw = {"w13_codes": torch.zeros(E, 2 * I, d // 2, dtype=torch.uint8, device="cuda"),
           "w13_scales": torch.zeros(E, 2 * I, d // 32, dtype=torch.uint8, device="cuda"),
           "w2_codes": torch.zeros(E, d, I // 2, dtype=torch.uint8, device="cuda"),
           "w2_scales": torch.zeros(E, d, I // 32, dtype=torch.uint8, device="cuda")}
    good = megamoe.MxWeights.prepare(raw)
    parts = [good.w13_codes, good.w13_scales, good.w2_codes, good.w2_scales]
    for i in range(4):
        for change, error in ((lambda t: t.cpu(), TypeError), (lambda t: t[:1], ValueError)):
            bad = list(parts)
            bad[i] = change(bad[i])
            with pytest.raises(error):
                megamoe.MxWeights(E, d, I, *bad)
    with pytest.raises(ValueError):
        megamoe.MxForward(good, 4, 2, device="cpu")
    fwd = megamoe.MxForward(good, 4, 2, device="cuda")
    assert fwd.ws.is_cuda


def test_status_words(cuda_lib):
    for status in (torch.zeros(1, dtype=torch.int32), torch.zeros(1, device="cuda"),
                   torch.zeros(1, dtype=torch.uint8, device="cuda")):
        with pytest.raises(TypeError):
            megamoe.quantize_mxfp4(_x(), status=status)
    with pytest.raises(ValueError):
        megamoe.quantize_mxfp4(_x(), status=torch.zeros(0, dtype=torch.int32, device="cuda"))


def test_one_row_of_any_stride(cuda_lib):
    """A row cut out of a matrix whose own rows are not on 16-byte boundaries."""
    x = torch.randn(1, K + 8, device="cuda").to(torch.bfloat16)
    odd = x.as_strided((1, K), (K + 1, 1))
    flat = odd.clone(memory_format=torch.contiguous_format)
    w = megamoe.MxLinearWeights.quantize(torch.randn(N, K, device="cuda"))
    out = torch.empty(1, N + 8, dtype=torch.bfloat16, device="cuda").as_strided((1, N), (N + 1, 1))
    want = megamoe.linear_mxfp4(flat, w)[0]
    assert torch.equal(megamoe.linear_mxfp4(odd, w)[0], want)
    assert torch.equal(megamoe.linear_mxfp4(flat, w, out=out)[0], want)
    for transpose in (False, True):
        for got, ref in zip(megamoe.quantize_mxfp4(odd, transpose),
                            megamoe.quantize_mxfp4(flat, transpose)):
            assert torch.equal(got, ref)
    g, m = torch.randn(1, N, device="cuda"), torch.randn(N, K, device="cuda")
    for got, ref in zip(megamoe.linear_mxfp4_backward(g, odd, m)[:2],
                        megamoe.linear_mxfp4_backward(g, flat, m)[:2]):
        assert torch.equal(got, ref)
