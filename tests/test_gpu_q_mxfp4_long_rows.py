"""Rows so long that offsets within an operand pass 32 bits.  Everything but the
last 1024 columns is zero, so the result is that of those columns alone."""

import pytest
import torch

from nvfp4_block_scaled_topk_gb300 import megamoe

pytestmark = pytest.mark.gpu

TAIL = 1024


def _codes(*shape):
    g = torch.Generator("cuda").manual_seed(len(shape))
    return torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)


def test_linear(cuda_lib):
    K, N = (1 << 29) + TAIL, 32
    codes = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    codes[:, -TAIL // 2:] = _codes(N, TAIL // 2)
    scales = torch.zeros(megamoe.mx_atom_bytes(N, K), dtype=torch.uint8, device="cuda")
    scales[-TAIL // 128 * 512:] = 127
    x = torch.zeros(1, K, dtype=torch.bfloat16, device="cuda")
    x[:, -TAIL:] = torch.randn(1, TAIL, device="cuda")
    out, ws = megamoe.linear_mxfp4(x, megamoe.MxLinearWeights(N, K, codes, scales),
                                   out_dtype=megamoe.EPI_F32)
    assert ws[:4].view(torch.int32).item() == 0
    xq = megamoe.dequantize_mxfp4(*megamoe.quantize_mxfp4(x[:, -TAIL:].contiguous()))
    wq = megamoe.dequantize_mxfp4(codes[:, -TAIL // 2:].contiguous(),
                                  torch.full((N, TAIL // 32), 127, dtype=torch.uint8, device="cuda"))
    a, b = xq.double(), wq.double()
    bound = (TAIL / 64 + 18) * 2.0 ** -23 * (a.abs() @ b.abs().t())
    assert ((out.double() - a @ b.t()).abs() <= bound).all() and out.any()


# tiles of 32 tokens, token-major tiles
@pytest.mark.parametrize("T", [1, 64])
def test_experts(cuda_lib, T):
    d, I = (1 << 24) + TAIL, 256
    tail = {"w13_codes": _codes(1, 2 * I, TAIL // 2), "w2_codes": _codes(1, TAIL, I // 2, 1)[..., 0]}
    tail["w13_scales"] = torch.full((1, 2 * I, TAIL // 32), 121, dtype=torch.uint8, device="cuda")
    tail["w2_scales"] = torch.full((1, TAIL, I // 32), 121, dtype=torch.uint8, device="cuda")
    raw = {"w13_codes": torch.zeros(1, 2 * I, d // 2, dtype=torch.uint8, device="cuda"),
           "w13_scales": torch.zeros(1, 2 * I, d // 32, dtype=torch.uint8, device="cuda"),
           "w2_codes": torch.zeros(1, d, I // 2, dtype=torch.uint8, device="cuda"),
           "w2_scales": torch.zeros(1, d, I // 32, dtype=torch.uint8, device="cuda")}
    raw["w13_codes"][..., -TAIL // 2:] = tail["w13_codes"]
    raw["w13_scales"][..., -TAIL // 32:] = tail["w13_scales"]
    raw["w2_codes"][:, -TAIL:] = tail["w2_codes"]
    raw["w2_scales"][:, -TAIL:] = tail["w2_scales"]
    x = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    x[:, -TAIL:] = torch.randn(T, TAIL, device="cuda") / 8
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    w = torch.ones(T, 1, device="cuda")
    weights = megamoe.MxWeights.prepare(raw)
    del raw
    fwd = megamoe.MxForward(weights, T, 1)
    out = fwd(x, ids, w)
    assert fwd.read_status() == 0
    short = megamoe.MxForward(megamoe.MxWeights.prepare(
        {n: t.contiguous() for n, t in tail.items()}), T, 1)
    want = short(x[:, -TAIL:].contiguous(), ids, w)
    # zeros in front of a sum change nothing in it
    assert want.any() and torch.equal(out[:, -TAIL:], want) and not out[:, :-TAIL].any()
