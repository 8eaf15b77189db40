"""The gated activation and its gradient where the exponential of the gate is smaller
than an fp32 number can be, and where a product of two factors is larger than one.

Each value is off by half a step of bf16 and by what fp32 adds: the exponential of half
the gate two units (2^-22 of the value), its square twice that and a rounding, the
reciprocal of 1 + e a unit and a rounding, four more products and a sum of halves: below
2^-20 of the value, for the gate's gradient of the larger of its two terms."""

import pytest
import torch

from nvfp4_block_scaled_topk_gb300 import megamoe

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
FAR = 2.0 ** -20


def _check(got, want, room):
    f = torch.finfo(got.dtype)
    assert torch.isfinite(want.to(got.dtype)).all()
    err = (got.double() - want).abs()
    bound = room + (want.abs() + room) * f.eps / 2 + f.smallest_normal * f.eps / 2
    bad = ~(err <= bound)
    assert not bad.any(), (got[bad][:4], want[bad][:4], bad.nonzero()[:4])


def _terms(gate, up, grad):
    """silu(g) u, the two terms of its gradient by g, and its gradient by u."""
    s, rest = torch.sigmoid(gate), torch.sigmoid(-gate)
    return gate * s * up, grad * up * s, grad * up * s * gate * rest, grad * gate * s


@pytest.mark.parametrize("up,grad", [(1e30, 1e-6), (-1e30, 3.0), (1.0, -1e30), (1e30, 1e30),
                                     (-3e38, 1e10), (1e-30, -1e34), (1e38, 1e-38), (0.5, 0.25)])
def test_gates_far_below_zero(cuda_lib, up, grad):
    gate = torch.linspace(-170, -60, 1024, dtype=torch.float64).to(BF).view(4, 256)
    up = (torch.linspace(0.5, 1, 256, dtype=torch.float64) * up).to(BF).expand(4, 256)
    grad = (torch.linspace(1, 0.5, 256, dtype=torch.float64) * grad).to(BF).expand(4, 256).contiguous()
    want, a, b, gu = _terms(gate.double(), up.double(), grad.double())
    fits = [t.abs() < 3e38 for t in (want, a, b, gu)]
    keep = (fits[0] & fits[1] & fits[2] & fits[3]).all(0)  # columns that bf16 holds
    assert keep.sum() >= 128
    x = torch.cat([gate, up], 1).cuda()
    out = megamoe.silu_mul(x).cpu()
    _check(out[:, keep], want[:, keep], FAR * want.abs()[:, keep])
    got = megamoe.silu_mul_backward(grad.cuda(), x).cpu()
    dg = got[:, :256]
    _check(dg[:, keep], (a + b)[:, keep], FAR * torch.maximum(a.abs(), b.abs())[:, keep])
    _check(got[:, 256:][:, keep], gu[:, keep], FAR * gu.abs()[:, keep])


def test_large_factors_around_zero(cuda_lib):
    """grad * up leaves fp32's range where the gate's factor brings it back."""
    gate = torch.linspace(-30, 30, 1024, dtype=torch.float64).to(BF).view(4, 256)
    for u, h in ((1e25, 1e15), (1e15, 1e25), (1e-30, 1e-9), (3e38, 0.5), (0.25, 3e38)):
        up = torch.full((4, 256), u, dtype=torch.float64).to(BF)
        grad = torch.full((4, 256), h, dtype=torch.float64).to(BF)
        want, a, b, gu = _terms(gate.double(), up.double(), grad.double())
        x = torch.cat([gate, up], 1).cuda()
        got = megamoe.silu_mul_backward(grad.cuda(), x).cpu()
        out = megamoe.silu_mul(x).cpu()
        for value, exact, room in ((out, want, want.abs()), (got[:, :256], a + b, torch.maximum(a.abs(), b.abs())),
                                   (got[:, 256:], gu, gu.abs())):
            ok = exact.abs() < 3e38
            _check(value[ok], exact[ok], FAR * room[ok])


def test_a_closed_gate_gives_zero(cuda_lib):
    x = torch.zeros((1, 16), dtype=BF, device="cuda")
    x[0, :8] = torch.tensor([-300.0, -1e4, -1e30, -3e38, 0.0, -0.0, 300.0, 1e30])
    x[0, 8:] = 2.0
    out = megamoe.silu_mul(x)[0]
    assert (out[:6] == 0).all() and out[6] == 600 and out[7] == 2 * x[0, 7]
    got = megamoe.silu_mul_backward(torch.ones((1, 8), dtype=BF, device="cuda"), x)[0]
    assert (got[:4] == 0).all() and (got[8:12] == 0).all()
    assert (got[4:6] == 1).all() and (got[6:8] == 2).all() and (got[14:] == x[0, 6:8]).all()
