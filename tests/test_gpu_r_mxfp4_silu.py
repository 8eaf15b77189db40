"""SiLU(gate) * up of the MXFP4 experts to fp32: values of h that lie 2^-19 to 2^-18
of themselves beside the edge of two codes fall on the right side of it, for gates
from -80 to 80.

Gate and up are exact: a token is 1 in the first element of every block of 32, so a
weight row with a digit of 0 to 3 there, on block scales 4^-j, gives any number of
2 d / 32 bits; of 16 blocks eleven are used, 22 bits, which fp32 sums hold.  The down
projection is the identity, so the output is the rounded h itself."""

import numpy as np
import pytest
import torch

from oracle import mxfp4 as mx
from nvfp4_block_scaled_topk_gb300 import megamoe

pytestmark = pytest.mark.gpu

D = I = 512
DIGITS = 11


def _rows(v):
    """Positive values in [1, 4) 2^e -> (codes [n, D], scale bytes [n, D / 32]) of rows
    whose first elements sum to them rounded to 22 bits, and those sums."""
    e = 2 * np.floor(np.log2(v) / 2)
    left = np.rint(v / np.exp2(e) * 4.0 ** (DIGITS - 1))
    codes = np.zeros((len(v), D), np.uint8)
    bytes_ = np.full((len(v), D // 32), 127, np.int64)
    total = left * 4.0 ** (1 - DIGITS) * np.exp2(e)
    of_digit = np.array([0, 2, 4, 5], np.uint8)  # E2M1 codes of 0, 1, 2, 3
    for j in range(DIGITS - 1, -1, -1):
        codes[:, 32 * j] = of_digit[(left % 4).astype(int)]
        bytes_[:, j] = 127 + e - 2 * j
        left = np.floor(left / 4)
    assert not left.any()
    return codes, bytes_.astype(np.uint8), total


def _silu(g):
    e = np.exp(-np.abs(g))
    return g * np.where(g >= 0, 1, e) / (1 + e)


# tiles of 32, of 64, token-major tiles, pairs of CTAs
@pytest.mark.parametrize("T", [3, 30, 90, 130])
@pytest.mark.parametrize("reach", [8.0, 80.0])
def test_values_beside_an_edge(cuda_lib, T, reach):
    rng = np.random.default_rng(int(reach))
    gate = np.exp(rng.uniform(np.log(0.25), np.log(reach), I)) * rng.choice([-1, 1], I)
    gate[::32] = np.abs(gate[::32])
    gc, gb, size = _rows(np.abs(gate))
    gate = np.sign(gate) * size
    # the first of a block of 32 sets its scale, 1: h = 4.5; the others lie at an edge
    edge = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], I)
    side = rng.choice([-1, 1], I) * 2.0 ** -rng.uniform(18, 19, I)
    edge[::32], side[::32] = 4.5, 0
    uc, ub, up = _rows(edge * (1 + side) / np.abs(_silu(gate)))
    h = _silu(gate) * up
    distance = np.abs(h) / edge - 1
    assert (np.abs(distance)[edge != 4.5] > 2.0 ** -20).all()
    gc |= (gate < 0).astype(np.uint8)[:, None] * 8 * (gc > 0)  # the gate's sign on its digits
    w13 = np.concatenate([mx.pack(gc), mx.pack(uc)])[None]
    s13 = np.concatenate([gb, ub])[None]
    eye, ones = np.zeros((1, D, I), np.uint8), np.full((1, D, I // 32), 127, np.uint8)
    eye[0, np.arange(D), np.arange(I)] = 2  # 1
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    weights = megamoe.MxWeights.prepare({"w13_codes": cuda(w13), "w13_scales": cuda(s13),
                                         "w2_codes": cuda(mx.pack(eye[0])[None]),
                                         "w2_scales": cuda(ones)})
    x = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    x[:, ::32] = 1
    out = megamoe.MxForward(weights, T, 1)(x, torch.zeros(T, 1, dtype=torch.int32, device="cuda"),
                                           torch.ones(T, 1, device="cuda"))
    want = mx.round_to_mx(h[None])[0]
    assert np.array_equal(out.double().cpu().numpy(), np.broadcast_to(want, (T, D)))
