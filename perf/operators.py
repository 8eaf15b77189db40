"""Cases of the scored router and the MXFP4 operators, their plain forms, and
their values in 64 bits.

Operators (``case["op"]``):

  route        scored router: sigmoid or softmax scores of every expert, a
               balance bias for the choice, groups of experts, top-k, weights
               from the unbiased scores
  route_grad   its gradient with respect to the logits
  quantize     MXFP4 quantisation (E2M1 elements, one power-of-two scale per
               32), along rows or along columns, returned as the values
  linear       y = Q(x) w^T with an MXFP4 weight (serving)
  linear_grad  dx and dw of the linear, every operand quantised along the
               dimension that its product sums over (training)
  experts      routed experts with MXFP4 weights: gate and up product,
               SiLU(gate) * up, requantised, down product, weighted sum

``own`` false: ``run`` computes them in elementary torch operations in 32
bits; true: through the package's entry points.
"""

import numpy as np
import torch

own = False

#: sums of two neighbouring decisions of the router closer than this (relative)
#: are not told apart by 32-bit scores; such tokens are drawn again
CONTESTED = 4e-6

ROUTE = {"k": 6, "score": "sigmoid", "bias": True, "n_group": 8, "topk_group": 4, "group_top": 2,
         "renormalize": True, "scale": 2.5, "masked": 0, "dtype": "float32"}


def listed():
    return [
        # one token of a decode step over 384 experts: latency is all
        {"name": "route one token", "op": "route", "T": 1, "E": 384, **ROUTE},
        # a prefill batch over 384 experts, five of them out of service
        {"name": "route prefill", "op": "route", "T": 16384, "E": 384, **ROUTE, "masked": 5},
        # a short ragged training batch, bf16 logits, softmax scores used as they are
        {"name": "route grad ragged", "op": "route_grad", "T": 1025, "E": 48, **ROUTE,
         "score": "softmax", "bias": False, "n_group": 1, "topk_group": 1, "renormalize": False,
         "scale": 1.0, "dtype": "bfloat16"},
        # a training batch
        {"name": "route grad batch", "op": "route_grad", "T": 16384, "E": 384, **ROUTE},
        # the activations of a decode step
        {"name": "quantize decode", "op": "quantize", "rows": 8, "K": 7168, "dtype": "bfloat16",
         "transpose": False},
        # activations of a training batch, an odd number of tokens, quantised along the tokens
        {"name": "quantize columns", "op": "quantize", "rows": 8195, "K": 7168,
         "dtype": "bfloat16", "transpose": True},
        # one token through a projection of a decode step
        {"name": "linear one token", "op": "linear", "T": 1, "K": 7168, "N": 1536},
        # a prefill batch through an up-projection
        {"name": "linear prefill", "op": "linear", "T": 4096, "K": 1536, "N": 24576},
        # a ragged fine-tuning batch
        {"name": "linear grad ragged", "op": "linear_grad", "T": 333, "K": 1536, "N": 2048},
        # a training batch
        {"name": "linear grad batch", "op": "linear_grad", "T": 8192, "K": 7168, "N": 2048},
        # a decode step over one slice of 48 experts
        {"name": "experts decode", "op": "experts", "T": 8, "E": 48, "k": 6, "d": 7168, "I": 2048,
         "skew": 0.0, "dropped": 0.0},
        # a prefill chunk of an odd size, uneven load, some slots without an expert
        {"name": "experts prefill", "op": "experts", "T": 2003, "E": 48, "k": 6, "d": 7168,
         "I": 2048, "skew": 0.3, "dropped": 0.02},
    ]


def _log_int(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi], never 3072."""
    n = int(round(lo * (hi / lo) ** rng.random()))
    return n + 1 if n == 3072 else min(max(n, lo), hi)


def _log_mult(rng, lo, hi, step):
    """A multiple of step spread over the logarithm of [lo, hi], never 3072."""
    n = max(lo // step, int(lo * (hi / lo) ** rng.random()) // step) * step
    return n + step if n == 3072 else n


def draw(rng):
    op = rng.choice(["route", "route_grad", "quantize", "linear", "linear_grad", "experts"])
    if op in ("route", "route_grad"):
        n_group = rng.choice([1, 1, 2, 4, 8])
        E = n_group * rng.randint(8, 384 // n_group)
        topk_group = rng.randint(max(1, n_group // 2), n_group)
        k = rng.randint(1, min(8, topk_group * (E // n_group)))
        return {"op": op, "T": _log_int(rng, 1, 16384), "E": E, "k": k,
                "score": rng.choice(["sigmoid", "softmax"]), "bias": rng.random() < 0.5,
                "n_group": n_group, "topk_group": topk_group, "group_top": rng.choice([1, 2]),
                "renormalize": rng.random() < 0.5, "scale": rng.choice([1.0, 2.5]),
                "masked": rng.choice([0, 0, rng.randint(1, 4)]),
                "dtype": rng.choice(["float32", "bfloat16"])}
    if op == "quantize":
        while True:
            c = {"op": op, "rows": _log_int(rng, 1, 16384), "K": _log_mult(rng, 64, 8192, 32),
                 "dtype": rng.choice(["bfloat16", "float16", "float32"]),
                 "transpose": rng.random() < 0.5}
            if c["rows"] * c["K"] <= 8195 * 7168 // (2 if c["dtype"] == "float32" else 1):
                return c
    if op in ("linear", "linear_grad"):
        most = 4096 * 1536 * 24576 if op == "linear" else 8192 * 7168 * 2048
        while True:
            c = {"op": op, "T": _log_int(rng, 1, 8192), "K": _log_mult(rng, 256, 8192, 32),
                 "N": _log_mult(rng, 256, 16384, 32)}
            if c["T"] * c["K"] * c["N"] <= most and c["K"] * c["N"] <= 1536 * 24576:
                return c
    while True:
        E = rng.choice([8, 16, 33, 48])
        c = {"op": op, "T": _log_int(rng, 1, 2003), "E": E, "k": rng.randint(1, min(8, E // 2)),
             "d": _log_mult(rng, 256, 7168, 256), "I": _log_mult(rng, 256, 2048, 256),
             "skew": rng.choice([0.0, 0.3]), "dropped": rng.choice([0.0, 0.02])}
        if c["T"] * c["k"] * c["d"] * c["I"] <= 2003 * 6 * 7168 * 2048 and c["I"] != 1536:
            return c


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, sigma, dtype):
    return torch.randn(shape, generator=g, device="cuda").mul_(sigma).to(dtype)


def _contested(case, logits, bias):
    """Rows of the logits whose choice of groups or experts hangs on two
    different scores that 32 bits may not tell apart (equal ones are ties)."""
    l = logits.double()
    dead = l == -torch.inf
    if case["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
    else:
        s = torch.exp(l - l.amax(1, keepdim=True))
        s = s / s.sum(1, keepdim=True)
    c = s if bias is None else s + bias.double()
    c = c.masked_fill(dead, -torch.inf)

    def close(v):  # of neighbours in descending order
        hi, lo = v[:, :-1], v[:, 1:]
        gap = hi - lo
        return ((gap > 0) & (gap < CONTESTED * torch.maximum(hi.abs(), lo.abs()))).any(1)

    bad = torch.zeros(l.shape[0], dtype=torch.bool, device=l.device)
    G = case["n_group"]
    if G > 1:
        top = torch.sort(c.view(-1, G, case["E"] // G), dim=2, descending=True)[0][..., :case["group_top"]]
        best = torch.where(top > -torch.inf, top, 0).sum(2)
        sorted_best, order = torch.sort(best, dim=1, descending=True, stable=True)
        bad |= close(sorted_best[:, case["topk_group"] - 1:case["topk_group"] + 1])
        kept = torch.zeros_like(best).scatter_(1, order[:, :case["topk_group"]], 1) > 0
        c = c.masked_fill(~kept.repeat_interleave(case["E"] // G, 1), -torch.inf)
    return bad | close(torch.sort(c, dim=1, descending=True)[0][:, :case["k"] + 1])


def _route_inputs(case, seed):
    g = _generator(seed)
    T, E, dtype = case["T"], case["E"], getattr(torch, case["dtype"])
    out = torch.randperm(E, generator=g, device="cuda")[:case["masked"]]
    # a balance bias moves by fixed steps
    bias = None
    if case["bias"]:
        bias = torch.randint(-24, 25, (E,), generator=g, device="cuda").float() / 1024

    def rows(n):
        l = _normal(g, (n, E), 1.5, dtype)
        l[:, out] = -torch.inf
        return l

    logits = rows(T)
    for _ in range(12):
        bad = _contested(case, logits, bias).nonzero().flatten()
        if not bad.numel():
            break
        logits[bad] = rows(bad.numel())
    return logits, bias, g


def _quantize_inputs(case, seed):
    g = _generator(seed)
    x = _normal(g, (case["rows"], case["K"]), 0.09, torch.float32)
    # a few large channels, as activations have
    loud = torch.randperm(case["K"], generator=g, device="cuda")[:max(1, case["K"] // 256)]
    x[:, loud] *= 16
    return x.to(getattr(torch, case["dtype"]))


def _linear_inputs(case, seed):
    g = _generator(seed)
    x = _normal(g, (case["T"], case["K"]), 0.09, torch.bfloat16)
    w = _normal(g, (case["N"], case["K"]), 0.02, torch.bfloat16)
    return x, w, g


def _experts_inputs(case, seed):
    g = _generator(seed)
    T, E, k, d, I = (case[n] for n in ("T", "E", "k", "d", "I"))
    x = _normal(g, (T, d), 0.09, torch.bfloat16)
    rank = torch.randperm(E, generator=g, device="cuda").float() + 1
    logits = torch.randn((T, E), generator=g, device="cuda") - case["skew"] * torch.log(rank)
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    weights = torch.exp(top[:, :k] - top[:, :1])
    weights = weights / weights.sum(1, keepdim=True)
    gone = torch.rand((T, k), generator=g, device="cuda") < case["dropped"]
    ids = ids[:, :k].masked_fill(gone, -1).to(torch.int32).contiguous()
    w13 = torch.empty((E, 2 * I, d // 2), dtype=torch.uint8, device="cuda")
    s13 = torch.empty((E, 2 * I, d // 32), dtype=torch.uint8, device="cuda")
    w2 = torch.empty((E, d, I // 2), dtype=torch.uint8, device="cuda")
    s2 = torch.empty((E, d, I // 32), dtype=torch.uint8, device="cuda")
    for e in range(E):
        w13[e], s13[e] = _encode(_normal(g, (2 * I, d), 0.02, torch.float32))
        w2[e], s2[e] = _encode(_normal(g, (d, I), 0.02, torch.float32))
    return x, ids, weights, {"w13_codes": w13, "w13_scales": s13, "w2_codes": w2, "w2_scales": s2}


def prepare(case, seed):
    op = case["op"]
    state = {"case": case}
    if op in ("route", "route_grad"):
        logits, bias, g = _route_inputs(case, seed)
        state |= {"logits": logits, "bias": bias}
        if op == "route_grad":
            state["ids"] = _route(case, logits, bias)[0]
            state["grad"] = torch.randn((case["T"], case["k"]), generator=g, device="cuda")
    elif op == "quantize":
        state["x"] = _quantize_inputs(case, seed)
    elif op == "linear":
        x, w, _ = _linear_inputs(case, seed)
        codes, scales = _encode(w.float())
        state |= {"x": x, "codes": codes, "scales": scales}
        if own:  # the weight as the program keeps it
            from nvfp4_block_scaled_topk_gb300 import megamoe
            state["weight"] = megamoe.MxLinearWeights.prepare(codes, scales)
    elif op == "linear_grad":
        x, w, g = _linear_inputs(case, seed)
        state |= {"x": x, "w": w,
                  "grad": _normal(g, (case["T"], case["N"]), 1e-3, torch.bfloat16)}
    else:
        x, ids, weights, experts = _experts_inputs(case, seed)
        load = torch.bincount(ids.flatten().clamp(min=0).long(), minlength=case["E"])
        state |= {"x": x, "ids": ids, "weights": weights, "experts": experts,
                  "room": int(load.max())}
        if own:  # the weights and the workspace as the program keeps them
            from nvfp4_block_scaled_topk_gb300 import megamoe
            state["forward"] = megamoe.MxForward(megamoe.MxWeights.prepare(experts), case["T"],
                                                 case["k"])
    return state


# --------------------------------------------------------------------------
# plain forms, 32 bits
# --------------------------------------------------------------------------
def _grid(x):
    """x [..., n] (n a multiple of 32) -> (element values on the E2M1 grid,
    scale exponents [..., n / 32]): exponent floor(log2(amax)) - 2, at least
    -127; elements to the nearest, ties to even, at most 6 in size."""
    b = x.unflatten(-1, (-1, 32))
    e = ((b.abs().amax(-1, keepdim=True).view(torch.int32) >> 23) - 129).clamp(min=-127)
    v = b / _power(e)
    size = v.abs()
    step = torch.where(size < 2, 0.5, torch.where(size < 4, 1.0, 2.0))
    q = torch.copysign((torch.round(size / step) * step).clamp(max=6), v)
    return q, e


def _power(e):
    """2^e, -127 <= e <= 127."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _mx(x):
    """x rounded to MXFP4 along its last dimension, as values."""
    q, e = _grid(x)
    return (q * _power(e)).flatten(-2)


def _mx_columns(x):
    """x [rows, n] -> [n, rows up to a multiple of 32], rounded along the rows."""
    t = x.t()
    return _mx(torch.nn.functional.pad(t, (0, -t.shape[1] % 32)).contiguous())


def _encode(x):
    """x [..., n] -> MXFP4 bytes: codes [..., n / 2] (the even element low) and
    scale bytes [..., n / 32]."""
    q, e = _grid(x)
    size = q.abs()
    code = torch.where(size < 2, size * 2, torch.where(size < 4, size + 2, size / 2 + 4))
    code = (code.to(torch.uint8) | (torch.signbit(q).to(torch.uint8) << 3)).flatten(-2)
    return code[..., ::2] | (code[..., 1::2] << 4), (e.squeeze(-1) + 127).to(torch.uint8)


def _decode(codes, scales):
    """The values of MXFP4 bytes."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    grid = torch.cat([grid, -grid])
    byte = torch.arange(256, device=codes.device)
    pair = torch.stack([grid[byte & 15], grid[byte >> 4]], 1)
    v = torch.index_select(pair, 0, codes.flatten().int())
    v = v.view(*scales.shape, 32) * _power(scales.int() - 127).unsqueeze(-1)
    return v.flatten(-2)


def _scores(case, logits):
    l = logits.float()
    dead = ~(l > -torch.inf)
    l = l.clamp(max=torch.finfo(torch.float32).max).masked_fill(dead, 0)
    if case["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
    else:
        s = torch.exp(l - l.masked_fill(dead, -torch.inf).amax(1, keepdim=True))
        s = s.masked_fill(dead, 0)
        s = s / s.sum(1, keepdim=True).clamp(min=1e-30)
    return s.masked_fill(dead, 0), dead


def _route(case, logits, bias):
    s, dead = _scores(case, logits)
    c = s if bias is None else s + bias
    c = c.masked_fill(dead | ~(c > -torch.inf), -torch.inf)
    G = case["n_group"]
    if G > 1:
        top = torch.sort(c.view(-1, G, case["E"] // G), dim=2, descending=True)[0][..., :case["group_top"]]
        best = torch.where(top > -torch.inf, top, 0).sum(2).masked_fill(top[..., 0] == -torch.inf, -torch.inf)
        kept = torch.sort(best, dim=1, descending=True, stable=True)[1][:, :case["topk_group"]]
        kept = torch.zeros_like(best).scatter_(1, kept, 1) > 0
        c = c.masked_fill(~kept.repeat_interleave(case["E"] // G, 1), -torch.inf)
    c, ids = torch.sort(c, dim=1, descending=True, stable=True)
    chosen = c[:, :case["k"]] > -torch.inf
    ids = ids[:, :case["k"]]
    w = s.gather(1, ids) * chosen
    if case["renormalize"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0)
    return ids.masked_fill(~chosen, -1).to(torch.int32), w * case["scale"]


def _route_grad(case, logits, ids, grad):
    s, _ = _scores(case, logits)
    chosen = ids >= 0
    at = ids.clamp(min=0).long()
    picked = s.gather(1, at) * chosen
    g = grad * case["scale"] * chosen
    if case["renormalize"]:
        total = picked.sum(1, keepdim=True)
        share = torch.where(total > 0, picked / total, 0)
        rest = g - (g * share).sum(1, keepdim=True)
        if case["score"] == "softmax":  # the sum over all experts cancels
            dl = share * rest
        else:
            dl = share * rest * (1 - picked)
        return torch.zeros_like(s).scatter_add_(1, at, dl * chosen).to(logits.dtype)
    if case["score"] == "sigmoid":
        dl = g * picked * (1 - picked)
        return torch.zeros_like(s).scatter_add_(1, at, dl * chosen).to(logits.dtype)
    full = torch.zeros_like(s).scatter_add_(1, at, g)
    return (s * (full - (g * picked).sum(1, keepdim=True))).to(logits.dtype)


def _experts(state):
    case, w = state["case"], state["experts"]
    E, I, room = case["E"], case["I"], state["room"]
    ids = state["ids"].long()
    # each expert's slots in order, in a table of the largest load's length
    slot = ids.flatten()
    order = torch.sort(torch.where(slot < 0, E, slot), stable=True)[1]
    expert = torch.where(slot < 0, E, slot)[order]
    count = torch.zeros(E + 1, dtype=torch.int64, device=slot.device)
    count = count.scatter_add_(0, expert, torch.ones_like(expert))
    place = torch.arange(len(order), device=slot.device) - (count.cumsum(0) - count)[expert]
    at = torch.empty_like(order).scatter_(0, order, expert * room + place.clamp(max=room - 1))
    table = torch.zeros(((E + 1) * room, case["d"]), device=slot.device)
    table[at] = _mx(state["x"].float()).repeat_interleave(case["k"], 0)
    table = table[:E * room].view(E, room, -1)
    h = table @ _decode(w["w13_codes"], w["w13_scales"]).transpose(1, 2)
    gate, up = h[..., :I], h[..., I:]
    h = _mx((gate / (1 + torch.exp(-gate)) * up).contiguous())
    y = h @ _decode(w["w2_codes"], w["w2_scales"]).transpose(1, 2)
    y = y.flatten(0, 1)[at.clamp(max=E * room - 1)].view(*ids.shape, -1)
    return (y * (state["weights"] * (ids >= 0)).unsqueeze(-1)).sum(1).to(torch.bfloat16)


def _plain(state):
    case = state["case"]
    op = case["op"]
    if op == "route":
        ids, w = _route(case, state["logits"], state["bias"])
        return {"ids": ids, "weights": w}
    if op == "route_grad":
        return {"grad_logits": _route_grad(case, state["logits"], state["ids"], state["grad"])}
    if op == "quantize":
        x = state["x"].float()
        return {"values": (_mx_columns(x) if case["transpose"] else _mx(x)).to(torch.bfloat16)}
    if op == "linear":
        y = _mx(state["x"].float()) @ _decode(state["codes"], state["scales"]).t()
        return {"out": y.to(torch.bfloat16)}
    if op == "linear_grad":
        x, w, dy = state["x"].float(), state["w"].float(), state["grad"].float()
        dx = _mx(dy) @ _mx_columns(w).t()
        return {"grad_x": dx.to(torch.bfloat16), "grad_w": _mx_columns(dy) @ _mx_columns(x).t()}
    return {"out": _experts(state)}


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def _own(state):
    from nvfp4_block_scaled_topk_gb300 import megamoe

    case = state["case"]
    op = case["op"]
    if op == "route":
        ids, w = megamoe.router_scored_topk(
            state["logits"], case["k"], case["score"], bias=state["bias"], n_group=case["n_group"],
            topk_group=case["topk_group"], group_top=case["group_top"],
            renormalize=case["renormalize"], scale=case["scale"])
        return {"ids": ids, "weights": w}
    if op == "route_grad":
        return {"grad_logits": megamoe.router_scored_topk_backward(
            state["logits"], state["ids"], state["grad"], case["score"],
            renormalize=case["renormalize"], scale=case["scale"])}
    if op == "quantize":
        codes, scales = megamoe.quantize_mxfp4(state["x"], transpose=case["transpose"])
        return {"values": megamoe.dequantize_mxfp4(codes, scales)}
    if op == "linear":
        return {"out": megamoe.linear_mxfp4(state["x"], state["weight"])[0]}
    if op == "linear_grad":
        dx, dw, _ = megamoe.linear_mxfp4_backward(state["grad"], state["x"], state["w"])
        return {"grad_x": dx, "grad_w": dw}
    return {"out": state["forward"](state["x"], state["ids"], state["weights"])}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    """Bytes: inputs once, outputs once. Operations: the products (or, for the
    router and the quantiser, a handful for each element)."""
    op = case["op"]
    if op in ("route", "route_grad"):
        size = 4 if case["dtype"] == "float32" else 2
        logits, slots = case["T"] * case["E"], case["T"] * case["k"]
        passes = 2 if op == "route_grad" else 1
        return {"bytes": logits * size * passes + slots * 8, "flops": logits * 6}
    if op == "quantize":
        n = case["rows"] * case["K"]
        return {"bytes": n * ((4 if case["dtype"] == "float32" else 2) + 2), "flops": n * 4}
    if op in ("linear", "linear_grad"):
        T, K, N = case["T"], case["K"], case["N"]
        if op == "linear":
            return {"bytes": 2 * T * K + N * K * 17 / 32 + 2 * T * N, "flops": 2 * T * K * N}
        return {"bytes": 4 * T * K + 6 * N * K + 2 * T * N, "flops": 4 * T * K * N}
    T, E, k, d, I = (case[n] for n in ("T", "E", "k", "d", "I"))
    active = E * (1 - (1 - k / E) ** T)
    return {"bytes": active * 3 * d * I * 17 / 32 + 4 * T * d + 8 * T * k,
            "flops": 6 * T * k * d * I * (1 - case["dropped"])}


# --------------------------------------------------------------------------
# the operators in 64 bits
# --------------------------------------------------------------------------
#: E2M1 values by code, and the midpoints between neighbours
_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_MIDDLE = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def _mx64(x):
    """x (64 bits) rounded to MXFP4 along the last dimension, the last block
    short where 32 does not divide it."""
    n = x.shape[-1]
    x = torch.cat([x, x.new_zeros(*x.shape[:-1], -n % 32)], -1)
    x = x.reshape(*x.shape[:-1], -1, 32)
    amax = x.abs().max(-1, keepdim=True)[0]
    e = torch.frexp(amax)[1].long() - 3  # amax in [2^(e+2), 2^(e+3))
    e = torch.where(amax == 0, -127, e).clamp(min=-127)
    unit = ((e + 1023) << 52).view(torch.float64)  # 2^e, exactly
    r = x.abs() / unit
    value = torch.zeros_like(r)
    for code, middle in enumerate(_MIDDLE):
        up = (r > middle) | ((r == middle) & (code % 2 == 1))  # a tie to the even code
        value = torch.where(up, _VALUES[code + 1], value)
    return (value * unit * torch.sign(x)).reshape(*x.shape[:-2], -1)


def _bytes64(codes, scales):
    value = torch.tensor(_VALUES + tuple(-v for v in _VALUES), dtype=torch.float64, device=codes.device)
    v = torch.stack([value[(codes % 16).long()], value[(codes // 16).long()]], -1).flatten(-2)
    return v * ((scales.long() + 896) << 52).view(torch.float64).repeat_interleave(32, -1)


def _scores64(case, logits):
    l = logits.double().cpu().numpy()
    with np.errstate(all="ignore"):
        if case["score"] == "sigmoid":
            return 1 / (1 + np.exp(-l))
        s = np.exp(l - l.max(1, keepdims=True))
        return s / s.sum(1, keepdims=True)


def _exact_route(case, seed):
    logits, bias, g = _route_inputs(case, seed)
    s = _scores64(case, logits)
    T, E, k, G = case["T"], case["E"], case["k"], case["n_group"]
    rows = np.arange(T)
    c = s + (0 if bias is None else bias.double().cpu().numpy())
    c[s == 0] = -np.inf
    groups = c.reshape(T, G, E // G)
    best = np.full((T, G), -np.inf)
    left = groups.copy()
    for j in range(case["group_top"]):
        at = left.argmax(2)
        v = np.take_along_axis(left, at[..., None], 2)[..., 0]
        best = np.where(v > -np.inf, np.where(best > -np.inf, best, 0) + v, best)
        np.put_along_axis(left, at[..., None], -np.inf, 2)
    kept = np.zeros((T, G), bool)
    for j in range(case["topk_group"]):
        at = best.argmax(1)
        kept[rows, at] |= best[rows, at] > -np.inf
        best[rows, at] = -np.inf
    c = np.where(kept[..., None], groups, -np.inf).reshape(T, E)
    ids = np.full((T, k), -1, np.int64)
    for j in range(k):
        at = c.argmax(1)
        ids[:, j] = np.where(c[rows, at] > -np.inf, at, -1)
        c[rows, at] = -np.inf
    w = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0)
    if case["renormalize"]:
        w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
    return logits, ids, w * case["scale"], s, g


def exact(case, seed):
    op = case["op"]
    if op == "route":
        _, ids, w, _, _ = _exact_route(case, seed)
        return {"ids": torch.from_numpy(ids).to(torch.int32), "weights": torch.from_numpy(w)}
    if op == "route_grad":
        logits, ids, w, s, g = _exact_route(case, seed)
        grad = torch.randn(ids.shape, generator=g, device="cuda").double().cpu().numpy()
        at = np.maximum(ids, 0)
        p = np.where(ids >= 0, np.take_along_axis(s, at, 1), 0)
        up = np.where(ids >= 0, grad * case["scale"], 0)
        if case["renormalize"]:  # w = scale p / sum p
            total = np.maximum(p.sum(1, keepdims=True), 1e-300)
            up = (up - (up * p).sum(1, keepdims=True) / total) / total
        ds = np.zeros_like(s)
        np.add.at(ds, (np.arange(case["T"])[:, None], at), up * (ids >= 0))
        if case["score"] == "sigmoid":
            dl = ds * s * (1 - s)
        else:
            dl = s * (ds - (ds * s).sum(1, keepdims=True))
        return {"grad_logits": torch.from_numpy(dl)}
    if op == "quantize":
        x = _quantize_inputs(case, seed).double()
        return {"values": _mx64(x.t() if case["transpose"] else x)}
    if op == "linear":
        x, w, _ = _linear_inputs(case, seed)
        return {"out": _mx64(x.double()) @ _mx64(w.double()).t()}
    if op == "linear_grad":
        x, w, g = _linear_inputs(case, seed)
        dy = _normal(g, (case["T"], case["N"]), 1e-3, torch.bfloat16).double()
        x, w = x.double(), w.double()
        return {"grad_x": _mx64(dy) @ _mx64(w.t()).t(), "grad_w": _mx64(dy.t()) @ _mx64(x.t()).t()}
    x, ids, weights, w = _experts_inputs(case, seed)
    xq = _mx64(x.double())
    out = torch.zeros_like(xq)
    for e in range(case["E"]):
        token, j = (ids == e).nonzero(as_tuple=True)
        if not len(token):
            continue
        h = xq[token] @ _bytes64(w["w13_codes"][e], w["w13_scales"][e]).t()
        gate, up = h[:, :case["I"]], h[:, case["I"]:]
        h = _mx64(gate / (1 + torch.exp(-gate)) * up)
        y = h @ _bytes64(w["w2_codes"][e], w["w2_scales"][e]).t()
        out.index_add_(0, token, y * weights[token, j].double().unsqueeze(1))
    return {"out": out}
