"""Waits that run out in the MXFP4 products: the kernel gives up as whole warps,
lets its copies land, reports MEGAMOE_DEV_TIMEOUT and returns, and the next call
is right."""

import numpy as np
import pytest
import torch

from nvfp4_block_scaled_topk_gb300 import megamoe

pytestmark = pytest.mark.gpu

LIMIT_NS = 100  # less than any load takes


def _normal(rows, cols, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, cols, generator=g) * scale).to(torch.bfloat16).cuda()


# both products in one launch of single CTAs; in clusters of their own; on pairs
@pytest.mark.parametrize("T,K,N", [(333, 512, 800), (7000, 256, 256), (2600, 4160, 2080)])
def test_gradients(cuda_lib, T, K, N):
    x, w, g = _normal(T, K, 1), _normal(N, K, 2, 0.02), _normal(T, N, 3)
    want_x, want_w, _ = megamoe.linear_mxfp4_backward(g, x, w)
    torch.cuda.synchronize()
    megamoe.set_wait_limit_ns(LIMIT_NS)
    try:
        _, _, ws = megamoe.linear_mxfp4_backward(g, x, w)
        torch.cuda.synchronize()
        assert ws[:4].view(torch.int32).item() == megamoe.DEV_TIMEOUT
    finally:
        megamoe.set_wait_limit_ns(0)
    got_x, got_w, ws = megamoe.linear_mxfp4_backward(g, x, w, ws=ws)
    assert ws[:4].view(torch.int32).item() == 0
    assert torch.equal(got_x, want_x) and torch.equal(got_w, want_w)


# tiles of 32 and 64 tokens, token-major tiles, pairs; K steps within the ring of
# stages (all loads are issued before anything gives up) and beyond it
@pytest.mark.parametrize("T,k", [(6, 3), (120, 3), (240, 3), (300, 3)])
@pytest.mark.parametrize("d", [256, 3328])
def test_experts(cuda_lib, T, k, d):
    E, I = 8, 256
    g = torch.Generator().manual_seed(d)

    def weight(rows, cols):
        w = torch.randn(E * rows, cols, generator=g).cuda() * 0.02
        codes, scales = megamoe.quantize_mxfp4(w)
        return codes.view(E, rows, -1), scales.view(E, rows, -1)

    w13, s13 = weight(2 * I, d)
    w2, s2 = weight(d, I)
    weights = megamoe.MxWeights.prepare({"w13_codes": w13, "w13_scales": s13, "w2_codes": w2,
                                         "w2_scales": s2})
    rng = np.random.default_rng(T)
    x = _normal(T, d, 5)
    ids = torch.tensor(np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)).cuda()
    w = torch.rand(T, k, generator=g).cuda()
    fwd = megamoe.MxForward(weights, T, k)
    want = fwd(x, ids, w).clone()
    assert fwd.read_status() == 0
    megamoe.set_wait_limit_ns(LIMIT_NS)
    try:
        fwd(x, ids, w)
        assert fwd.read_status() & megamoe.DEV_TIMEOUT
    finally:
        megamoe.set_wait_limit_ns(0)
    assert torch.equal(fwd(x, ids, w), want)
    assert fwd.read_status() == 0
