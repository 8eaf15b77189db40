"""MXFP4 products that keep their persistent kernels going: more tiles than CTAs
(or pairs of CTAs) and more K steps than stages, so that rings wrap, accumulators
are handed back and one tile's stores meet the next one's products.

The reference is fp32 products of the decoded values on the GPU (TF32 off), whose
own sums carry the same error bound.  The experts' intermediate is decided on such
sums, so a value on the edge of two codes may fall either way; the framework's bound
for a forward (helpers.py) holds."""

import numpy as np
import pytest
import torch

from nvfp4_block_scaled_topk_gb300 import megamoe
from helpers import assert_close_bf16

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
D = I = 3328  # 13 K steps, 26 tiles of 128


def _mx(x, transpose=False):
    return megamoe.dequantize_mxfp4(*megamoe.quantize_mxfp4(x, transpose=transpose),
                                    dtype=torch.float32)


def _experts(E, seed):
    g = torch.Generator("cuda").manual_seed(seed)

    def weight(rows, cols):
        w = torch.randn(E * rows, cols, generator=g, device="cuda") * 0.02
        codes, scales = megamoe.quantize_mxfp4(w)
        return codes.view(E, rows, -1), scales.view(E, rows, -1)

    w13, s13 = weight(2 * I, D)
    w2, s2 = weight(D, I)
    return {"w13_codes": w13, "w13_scales": s13, "w2_codes": w2, "w2_scales": s2}


def _reference(x, ids, w, raw):
    xq = _mx(x)
    out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    for e in range(raw["w13_codes"].shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not len(t):
            continue
        w13 = megamoe.dequantize_mxfp4(raw["w13_codes"][e], raw["w13_scales"][e], torch.float32)
        w2 = megamoe.dequantize_mxfp4(raw["w2_codes"][e], raw["w2_scales"][e], torch.float32)
        h = xq[t] @ w13.t()
        gate, up = h[:, :I], h[:, I:]
        y = _mx((gate / (1 + torch.exp(-gate)) * up).contiguous()) @ w2.t()
        out.index_add_(0, t, y.double() * w[t, j, None].double())
    return out


# rows an expert on average: tiles of 32 tokens, of 64, token-major tiles, pairs
@pytest.mark.parametrize("E,T,k", [(24, 200, 2), (24, 500, 2), (24, 1100, 2), (8, 2100, 2)])
def test_experts(cuda_lib, E, T, k):
    raw = _experts(E, E)
    rng = np.random.default_rng(T)
    x = torch.tensor(rng.standard_normal((T, D)) * 0.1, dtype=torch.bfloat16).cuda()
    # uneven loads, one expert without rows, some slots without an expert
    score = rng.gumbel(size=(T, E)) - 0.4 * np.log(np.arange(E) + 1)
    score[:, E // 2] = -np.inf
    ids = np.argsort(-score, axis=1)[:, :k].astype(np.int32)
    ids[rng.random((T, k)) < 0.02] = -1
    ids = torch.from_numpy(ids).cuda()
    w = torch.tensor(rng.random((T, k)) + 0.1, dtype=torch.float32).cuda()
    fwd = megamoe.MxForward(megamoe.MxWeights.prepare(raw), T, k)
    out = fwd(x, ids, w).clone()
    assert fwd.read_status() == 0
    want = _reference(x, ids, w, raw)
    assert_close_bf16(out.double().cpu().numpy(), want.cpu().numpy(), what="mxfp4 experts")
    for _ in range(3):
        assert torch.equal(fwd(x, ids, w), out)


# one launch for both gradients, of which one splits its tiles over clusters (of 8,
# 4 and 2 CTAs; of 8 and first in the launch) and the other does not: 110 tiles of
# the first take 112 blocks; then one gradient on pairs, the other beside it
@pytest.mark.parametrize("T,K,N", [(7000, 256, 256), (6200, 512, 640), (7200, 512, 1280),
                                   (333, 128, 8192), (700, 1280, 4096)])
def test_gradients(cuda_lib, T, K, N):
    g = torch.Generator("cuda").manual_seed(T)
    x = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(N, K, generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn(T, N, generator=g, device="cuda").to(torch.bfloat16)
    for gx_dt, gw_dt in ((torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)):
        gx, gw, ws = megamoe.linear_mxfp4_backward(dy, x, w, gx_dt, gw_dt)
        assert ws[:4].view(torch.int32).item() == 0
        for got, a, b in ((gx, _mx(dy), _mx(w, True)), (gw, _mx(dy, True), _mx(x, True))):
            want = a @ b.t()
            bound = 2 * (a.shape[1] / 64 + 18) * U * (a.abs() @ b.abs().t())
            if got.dtype == torch.bfloat16:
                bound = bound + 2.0 ** -8 * (want.abs() + bound)
            assert ((got.float() - want).abs() <= bound).all()
        again = megamoe.linear_mxfp4_backward(dy, x, w, gx_dt, gw_dt, ws=ws)
        assert torch.equal(again[0], gx) and torch.equal(again[1], gw)


# pairs: 6 stages and 5, more tiles than pairs, the accumulators in turn
@pytest.mark.parametrize("T,K,N", [(5000, 1536, 4128), (5000, 3360, 4128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear(cuda_lib, T, K, N, dtype):
    g = torch.Generator("cuda").manual_seed(K)
    x = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(N, K, generator=g, device="cuda").to(torch.bfloat16)
    weights = megamoe.MxLinearWeights.quantize(w)
    epi = megamoe.EPI_F32 if dtype == torch.float32 else megamoe.EPI_BF16
    out, ws = megamoe.linear_mxfp4(x, weights, out_dtype=epi)
    a, b = _mx(x), _mx(w)
    want = a @ b.t()
    bound = 2 * (K / 64 + 18) * U * (a.abs() @ b.abs().t())
    if dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (want.abs() + bound)
    assert ((out.float() - want).abs() <= bound).all()
    for _ in range(3):
        assert torch.equal(megamoe.linear_mxfp4(x, weights, out_dtype=epi, ws=ws)[0], out)
