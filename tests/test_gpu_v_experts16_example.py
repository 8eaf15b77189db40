"""The 16-bit experts' example runs, and its gradients are those of its forward pass."""

import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(cuda_lib):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import experts16_layer
    finally:
        sys.path.pop(0)
    return experts16_layer


def test_runs(example):
    losses, worst, status = example.main()
    assert all(math.isfinite(v) for v in losses) and status == 0
    # sums below 2^24 are exact whichever kernel takes them
    assert worst == 0


def test_gradients(example):
    """Against differences: the change of sum(out * g) along a direction of the weights,
    in a layer whose every value is off by 2^-8 of itself at most."""
    x, logits, w13, w2, g = example.inputs(3)
    out, saved = example.forward(x, logits, w13, w2)
    grads = example.backward(g, saved)
    # 64-bit layer with the same choice of experts
    ids = saved[1].long()

    def layer(x, logits, w13, w2):
        s = torch.sigmoid(logits).gather(1, ids)
        s = s / s.sum(1, keepdim=True)
        total = 0
        for j in range(example.K_TOP):
            a = torch.einsum("td,tnd->tn", x, w13[ids[:, j]])
            h = a[:, :example.I] * torch.sigmoid(a[:, :example.I]) * a[:, example.I:]
            total = total + torch.einsum("ti,tdi->td", h, w2[ids[:, j]]) * s[:, j:j + 1]
        return total

    at = [t.double() for t in (x, logits, w13, w2)]
    want = layer(*at)
    assert ((out.double() - want).norm() / want.norm()) < 4 * 2.0 ** -8
    gen = torch.Generator(device="cuda").manual_seed(9)
    for i, grad in enumerate(grads):
        d = torch.randn(at[i].shape, generator=gen, device="cuda", dtype=torch.float64)
        eps = 1e-4
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + eps * d, at[i] - eps * d
        diff = ((layer(*up) - layer(*down)) * g.double()).sum() / (2 * eps)
        got = (grad.double() * d).sum()
        # the gradient's errors are at most 6 * 2^-8 of its norm (six roundings to bf16
        # between input and gradient), and lie along a random direction like itself; five
        # standard deviations of |grad| |d| / sqrt(n)
        room = 5 * 6 * 2.0 ** -8 * grad.double().norm()
        assert (got - diff).abs() < room
