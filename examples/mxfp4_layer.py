"""A routed-expert layer and a linear in MXFP4, as a program uses them.

  * serving: a prompt, then single tokens, through the scored router (sigmoid
    scores, balance bias, groups) and MXFP4 experts in one call each;
  * training: a few steps of the router's projection and of an MXFP4 linear
    against fixed targets; the linear's master weight is quantised anew at every
    step, its gradients are products of MXFP4 operands, the router's gradient
    goes through its weights.

Run on a GPU:  python examples/mxfp4_layer.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from nvfp4_block_scaled_topk_gb300 import megamoe  # noqa: E402

E, K_TOP, D, I = 32, 4, 512, 256
ROUTE = dict(score="sigmoid", n_group=4, topk_group=2, group_top=2, renormalize=True, scale=2.5)


def make_experts(g):
    """Row-major MXFP4 expert weights, quantised from normal draws."""
    raw = {}
    for name, rows, cols in (("w13", 2 * I, D), ("w2", D, I)):
        w = torch.randn(E * rows, cols, generator=g, device="cuda") * 0.05
        codes, scales = megamoe.quantize_mxfp4(w)
        raw[name + "_codes"] = codes.view(E, rows, cols // 2)
        raw[name + "_scales"] = scales.view(E, rows, cols // 32)
    return megamoe.MxWeights.prepare(raw)


def serve(g):
    experts = make_experts(g)
    router = torch.randn(E, D, generator=g, device="cuda").bfloat16() / D ** 0.5
    bias = torch.zeros(E, device="cuda")
    prompt = torch.randn(300, D, generator=g, device="cuda").bfloat16()
    layer = megamoe.MxForward(experts, T=300, k=K_TOP)
    out = layer.from_logits(prompt, prompt @ router.t(), bias=bias, **ROUTE)
    print(f"prompt of {len(prompt)} tokens: output rms {out.float().square().mean().sqrt():.3f}, "
          f"status {layer.read_status()}")
    step = megamoe.MxForward(experts, T=1, k=K_TOP)
    worst = 0.0
    for t in (0, 17, 299):  # the same tokens one at a time
        x = prompt[t:t + 1]
        one = step.from_logits(x, x @ router.t(), bias=bias, **ROUTE)
        worst = max(worst, ((one - out[t]).float().norm() / out[t].float().norm()).item())
    print(f"single tokens against the prompt's rows: relative difference {worst:.1e}")
    # the balance bias moves by fixed steps against the load
    ids, _ = megamoe.router_scored_topk(prompt @ router.t(), K_TOP, bias=bias, **ROUTE)
    load = torch.bincount(ids.flatten().long(), minlength=E).float()
    bias += 1e-3 * torch.sign(load.mean() - load)
    return worst


def train(g, steps=60):
    x = torch.randn(1024, D, generator=g, device="cuda").bfloat16()
    target = torch.randn(D, D, generator=g, device="cuda") / D ** 0.5
    want = x.float() @ target.t()
    w = torch.zeros(D, D, device="cuda")
    losses = []
    for _ in range(steps):
        y, _ = megamoe.linear_mxfp4(x, megamoe.MxLinearWeights.quantize(w), megamoe.EPI_F32)
        error = y - want
        losses.append(error.square().mean().item())
        _, grad_w, _ = megamoe.linear_mxfp4_backward(error, x, w, need_x=False)
        w -= 0.3 / len(x) * grad_w  # below 2 over the largest curvature, 2.9
    print(f"linear: mean squared error {losses[0]:.3f} -> {losses[-1]:.3f} in {steps} steps")

    # the router learns to give its first expert's share to one side
    r = torch.randn(E, D, generator=g, device="cuda") * 0.02
    shares = []
    for _ in range(steps):
        logits = x.float() @ r.t()
        ids, weights = megamoe.router_scored_topk(logits, K_TOP, **ROUTE)
        shares.append(weights[:, 0].mean().item())
        grad = torch.zeros_like(weights)
        grad[:, 0] = -1.0 / len(x)  # more weight on the first choice
        grad_logits = megamoe.router_scored_topk_backward(logits, ids, grad, ROUTE["score"],
                                                          ROUTE["renormalize"], ROUTE["scale"])
        r -= 0.5 * (grad_logits.t() @ x.float())
    print(f"router: first choice's weight {shares[0]:.3f} -> {shares[-1]:.3f} in {steps} steps")
    return losses, shares


def main():
    g = torch.Generator(device="cuda").manual_seed(0)
    return serve(g), *train(g)


if __name__ == "__main__":
    main()
