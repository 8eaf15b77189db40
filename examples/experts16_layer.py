"""A routed-expert layer in 16 bits, trained and then served in 8-bit integers, as a
program uses it.

  * training: scored router, rows into the experts' order, gate and up products,
    SiLU(gate) * up, down products, weighted sum; back through all of them to the
    gradients of the tokens, of every expert's weights and of the router's logits;
    a few steps of plain gradient descent against fixed targets;
  * serving: a dense projection behind the layer, quantised once to 8-bit integers,
    for the whole batch and for single tokens.

Run on a GPU:  python examples/experts16_layer.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from nvfp4_block_scaled_topk_gb300 import megamoe  # noqa: E402

T, E, K_TOP, D, I = 200, 8, 2, 256, 136


def forward(x, logits, w13, w2):
    """The layer's output and what its backward pass needs."""
    ids, weights = megamoe.router_scored_topk(logits, K_TOP)
    route = megamoe.route_permute(ids, E)
    offsets, slots = route["offsets"], route["slot_dst"].view(T, K_TOP)
    live = offsets[E:]  # rows in use
    rows = megamoe.gather_rows(x, route["row_src"], K_TOP)
    a = megamoe.grouped_linear(rows, w13, offsets)
    h = megamoe.silu_mul(a, live_rows=live)
    y = megamoe.grouped_linear(h, w2, offsets)
    out = megamoe.combine_rows(y, slots, weights)
    return out, (logits, ids, weights, offsets, slots, live, rows, a, h, y, w13, w2)


def backward(grad, saved):
    """Gradients of x, logits, w13 and w2 (the weights' in fp32)."""
    logits, ids, weights, offsets, slots, live, rows, a, h, y, w13, w2 = saved
    grad_y, grad_weights = megamoe.combine_rows_backward(grad, y, slots, weights)
    grad_h, grad_w2 = megamoe.grouped_linear_backward(grad_y, h, w2, offsets)
    grad_a = megamoe.silu_mul_backward(grad_h, a, live_rows=live)
    grad_rows, grad_w13 = megamoe.grouped_linear_backward(grad_a, rows, w13, offsets)
    grad_x = megamoe.combine_rows(grad_rows, slots)
    return grad_x, megamoe.router_scored_topk_backward(logits, ids, grad_weights), grad_w13, grad_w2


def inputs(seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    return (normal(T, D).bfloat16(), normal(T, E), (normal(E, 2 * I, D) / 16).bfloat16(),
            (normal(E, D, I) / 12).bfloat16(), normal(T, D).bfloat16())


def train(steps=20, rate=0.01):
    x, logits, w13, w2, target = inputs()
    masters = [w13.float(), w2.float()]
    losses = []
    for _ in range(steps):
        out, saved = forward(x, logits, masters[0].bfloat16(), masters[1].bfloat16())
        miss = out.float() - target.float()
        losses.append(miss.square().mean().item())
        grads = backward((2 * miss / T).bfloat16(), saved)
        for m, g in zip(masters, grads[2:]):
            m -= rate * g
    return losses


def serve():
    """The largest relative difference between a token alone and in the batch."""
    x, logits, w13, w2, _ = inputs()
    g = torch.Generator(device="cuda").manual_seed(1)
    project = megamoe.Int8LinearWeights.quantize(torch.randn(512, D, generator=g, device="cuda") / 16)
    hidden, _ = forward(x, logits, w13, w2)
    all_, ws = megamoe.linear_int8(hidden, project)
    worst = 0.0
    for t in (0, 17, T - 1):
        one, _ = megamoe.linear_int8(hidden[t:t + 1], project)
        worst = max(worst, ((one[0] - all_[t]).float().norm() / all_[t].float().norm()).item())
    return worst, int(ws[:4].view(torch.int32))


def main():
    losses = train()
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    worst, status = serve()
    print(f"8-bit projection: a token alone differs from the batch by {worst:.1e}, status {status}")
    return losses, worst, status


if __name__ == "__main__":
    main()
