"""Cases of the operators of routed experts in 16 bits and of the 8-bit integer
linear, their plain forms, and their values in 64 bits.

Operators (``case["op"]``):

  grouped       products grouped by expert: out[r] = x[r] w[e(r)]^T for rows in
                the order of their experts, ragged row counts
  grouped_grad  its gradients with respect to the rows and to every expert's weight
  int8          y = (q_x q_w^T) s_x s_w: activations quantised to 8-bit integers
                with a scale for each token, weights with one for each channel
  silu          the gated activation between an expert's two products
  silu_grad     its gradient
  gather        tokens copied into the experts' row order
  combine       the weighted sum of each token's rows
  combine_grad  its gradients with respect to the rows and to the weights

``own`` false: ``run`` computes them in elementary torch operations in 32
bits; true: through the package's entry points.
"""

import torch

own = False


def listed():
    return [
        # gate and up products of a decode step over one slice of 48 experts: a
        # row or two an expert
        {"name": "grouped decode", "op": "grouped", "T": 8, "E": 48, "k": 6, "K": 7168, "N": 4096,
         "skew": 0.0, "dropped": 0.0, "dtype": "bfloat16", "out": "bfloat16"},
        # down products of a prefill chunk of an odd size, uneven load, some slots
        # without an expert
        {"name": "grouped prefill", "op": "grouped", "T": 2003, "E": 48, "k": 6, "K": 2048,
         "N": 7168, "skew": 0.3, "dropped": 0.02, "dtype": "bfloat16", "out": "bfloat16"},
        # a short training batch of small experts, very uneven, sizes that end inside tiles
        {"name": "grouped grad ragged", "op": "grouped_grad", "T": 333, "E": 16, "k": 4, "K": 1000,
         "N": 520, "skew": 0.8, "dropped": 0.02, "dtype": "float16", "out": "float32"},
        # a training batch of eight large experts
        {"name": "grouped grad batch", "op": "grouped_grad", "T": 8192, "E": 8, "k": 2, "K": 2048,
         "N": 7168, "skew": 0.3, "dropped": 0.0, "dtype": "bfloat16", "out": "float32"},
        # a projection of one token: the weights' bytes are all
        {"name": "int8 one token", "op": "int8", "T": 1, "K": 1536, "N": 24576,
         "dtype": "bfloat16", "out": "bfloat16"},
        # sizes that end inside tiles
        {"name": "int8 ragged", "op": "int8", "T": 333, "K": 1552, "N": 2056, "dtype": "float16",
         "out": "float32"},
        # a long prefill batch
        {"name": "int8 batch", "op": "int8", "T": 8192, "K": 7168, "N": 2048, "dtype": "bfloat16",
         "out": "bfloat16"},
        # the activation of a decode step's 48 rows
        {"name": "silu decode", "op": "silu", "rows": 48, "I": 2048, "dtype": "bfloat16"},
        # and its gradient in a training batch of 8192 tokens of six slots
        {"name": "silu grad batch", "op": "silu_grad", "rows": 49152, "I": 2048,
         "dtype": "bfloat16"},
        # a prefill chunk's tokens into the experts' order
        {"name": "gather prefill", "op": "gather", "T": 2003, "E": 48, "k": 6, "d": 7168,
         "skew": 0.3, "dropped": 0.02, "dtype": "bfloat16"},
        # the end of a decode step
        {"name": "combine decode", "op": "combine", "T": 8, "E": 48, "k": 6, "d": 7168, "skew": 0.0,
         "dropped": 0.0, "dtype": "bfloat16"},
        # the first step of a training batch's backward pass
        {"name": "combine grad batch", "op": "combine_grad", "T": 8192, "E": 48, "k": 6, "d": 7168,
         "skew": 0.3, "dropped": 0.02, "dtype": "bfloat16"},
    ]


def _log_int(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(max(int(round(lo * (hi / lo) ** rng.random())), lo), hi)


def _log_mult(rng, lo, hi, step):
    """A multiple of step spread over the logarithm of [lo, hi]."""
    return max(lo // step, int(lo * (hi / lo) ** rng.random()) // step) * step


def _load(rng, T):
    """Sizes of a routed batch."""
    E = rng.choice([1, 8, 16, 33, 48])
    return {"T": _log_int(rng, 1, T), "E": E, "k": rng.randint(1, min(8, E)),
            "skew": rng.choice([0.0, 0.3, 0.8]), "dropped": rng.choice([0.0, 0.02])}


def draw(rng):
    op = rng.choice(["grouped", "grouped", "grouped_grad", "grouped_grad", "int8", "int8", "silu",
                     "silu_grad", "gather", "combine", "combine_grad"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float16"])
    if op in ("grouped", "grouped_grad"):
        while True:
            c = {"op": op, **_load(rng, 8192), "K": _log_mult(rng, 64, 7168, 8),
                 "N": _log_mult(rng, 64, 7168, 8), "dtype": dtype,
                 "out": rng.choice([dtype, "float32"])}
            rows, weight = c["T"] * c["k"], c["K"] * c["N"]
            if op == "grouped" and rows * weight <= 12018 * 2048 * 7168 and c["E"] * weight <= 48 * 2048 * 7168:
                return c
            if op == "grouped_grad" and rows * weight <= 16384 * 2048 * 7168 and c["E"] * weight <= 8 * 2048 * 7168:
                return c
    if op == "int8":
        while True:
            c = {"op": op, "T": _log_int(rng, 1, 8192), "K": _log_mult(rng, 64, 8192, 16),
                 "N": _log_mult(rng, 64, 24576, 8),
                 "dtype": rng.choice(["bfloat16", "bfloat16", "float16", "float32"]),
                 "out": rng.choice(["bfloat16", "float32"])}
            if c["T"] * c["K"] * c["N"] <= 8192 * 7168 * 2048 and c["K"] * c["N"] <= 1536 * 24576:
                return c
    if op in ("silu", "silu_grad"):
        while True:
            c = {"op": op, "rows": _log_int(rng, 1, 49152), "I": _log_mult(rng, 64, 8192, 8),
                 "dtype": dtype}
            if c["rows"] * c["I"] <= 49152 * 2048:
                return c
    return {"op": op, **_load(rng, 8192), "d": _log_mult(rng, 64, 7168, 8), "dtype": dtype}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, sigma, dtype):
    return torch.randn(shape, generator=g, device="cuda").mul_(sigma).to(dtype)


def _type(name):
    return getattr(torch, name)


def _routing(case, g):
    """Expert of every slot, and the slots in the experts' order: offsets
    [E + 1], row_src (a row's slot) and slot_dst (a slot's row, -1 without one)."""
    T, E, k = case["T"], case["E"], case["k"]
    rank = torch.randperm(E, generator=g, device="cuda").float() + 1
    score = torch.randn((T, E), generator=g, device="cuda") - case["skew"] * torch.log(rank)
    ids = torch.sort(score, dim=1, descending=True, stable=True)[1][:, :k]
    slot = ids.flatten()
    slot[torch.randperm(T * k, generator=g, device="cuda")[:int(T * k * case["dropped"])]] = E
    order = torch.sort(slot, stable=True)[1]
    count = torch.bincount(slot, minlength=E + 1)[:E]
    live = int(count.sum())
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = count.cumsum(0)
    src = order[:live]
    dst = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    dst[src] = torch.arange(live, dtype=torch.int32, device="cuda")
    expert = slot[src]
    return {"offsets": offsets, "row_src": src.to(torch.int32), "slot_dst": dst.view(T, k),
            "expert": expert, "room": int(count.max()), "live": live}


def _experts(case, g):
    """[E, N, K] weights, made expert by expert."""
    w = torch.empty((case["E"], case["N"], case["K"]), dtype=_type(case["dtype"]), device="cuda")
    for e in range(case["E"]):
        w[e] = _normal(g, (case["N"], case["K"]), 0.02, w.dtype)
    return w


def _grouped_inputs(case, seed):
    g = _generator(seed)
    r = _routing(case, g)
    dtype = _type(case["dtype"])
    r["x"] = _normal(g, (r["live"], case["K"]), 0.5, dtype)
    r["w"] = _experts(case, g)
    if case["op"] == "grouped_grad":
        r["grad"] = _normal(g, (r["live"], case["N"]), 0.02, dtype)
    return r


def _int8_inputs(case, seed):
    g = _generator(seed)
    x = _normal(g, (case["T"], case["K"]), 0.09, torch.float32)
    # a few large channels, as activations have
    loud = torch.randperm(case["K"], generator=g, device="cuda")[:max(1, case["K"] // 256)]
    x[:, loud] *= 16
    w = torch.randint(-127, 128, (case["N"], case["K"]), generator=g, device="cuda",
                      dtype=torch.int8)
    s = torch.rand(case["N"], generator=g, device="cuda") * 2e-4 + 1e-4
    return {"x": x.to(_type(case["dtype"])), "codes": w, "scales": s}


def _silu_inputs(case, seed):
    g = _generator(seed)
    dtype = _type(case["dtype"])
    r = {"a": _normal(g, (case["rows"], 2 * case["I"]), 2.0, dtype)}
    if case["op"] == "silu_grad":
        r["grad"] = _normal(g, (case["rows"], case["I"]), 0.02, dtype)
    return r


def _rows_inputs(case, seed):
    g = _generator(seed)
    r = _routing(case, g)
    dtype = _type(case["dtype"])
    if case["op"] == "gather":
        r["x"] = _normal(g, (case["T"], case["d"]), 0.5, dtype)
        return r
    r["y"] = _normal(g, (r["live"], case["d"]), 0.5, dtype)
    weights = torch.exp(torch.randn((case["T"], case["k"]), generator=g, device="cuda"))
    r["weights"] = weights / weights.sum(1, keepdim=True)
    if case["op"] == "combine_grad":
        r["grad"] = _normal(g, (case["T"], case["d"]), 0.02, dtype)
    return r


def _inputs(case, seed):
    op = case["op"]
    if op in ("grouped", "grouped_grad"):
        return _grouped_inputs(case, seed)
    if op == "int8":
        return _int8_inputs(case, seed)
    return _silu_inputs(case, seed) if op in ("silu", "silu_grad") else _rows_inputs(case, seed)


def prepare(case, seed):
    state = {"case": case, **_inputs(case, seed)}
    if own and case["op"] == "int8":  # the weight as the program keeps it
        from nvfp4_block_scaled_topk_gb300 import megamoe
        state["weight"] = megamoe.Int8LinearWeights(case["N"], case["K"], state["codes"],
                                                    state["scales"])
    return state


# --------------------------------------------------------------------------
# plain forms, 32 bits
# --------------------------------------------------------------------------
def _table(state, rows):
    """Rows in experts' order -> [E, room, columns], zeros behind an expert's
    last, and the place of each row in it."""
    E, room, expert = state["case"]["E"], state["room"], state["expert"]
    first = state["offsets"].long()[expert]
    at = expert * room + torch.arange(len(rows), device=rows.device) - first
    table = torch.zeros((E * room, rows.shape[1]), device=rows.device)
    table[at] = rows.float()
    return table.view(E, room, -1), at


def _codes(x):
    """8-bit integers of each row and its scale; the choice of an integer is
    taken in 64 bits."""
    amax = x.abs().amax(1, keepdim=True)
    q = torch.round(x.double() * 127 / torch.where(amax > 0, amax, 1).double())
    return q.float(), amax.float() / 127


def _silu_grad(grad, a):
    gate, up = a.float().chunk(2, 1)
    s = 1 / (1 + torch.exp(-gate))
    grad = grad.float()
    return torch.cat([grad * up * s * (1 + gate * (1 - s)), grad * gate * s], 1)


def _plain(state):
    case = state["case"]
    op = case["op"]
    if op == "grouped":
        x, at = _table(state, state["x"])
        y = x @ state["w"].float().transpose(1, 2)
        return {"out": y.flatten(0, 1)[at].to(_type(case["out"]))}
    if op == "grouped_grad":
        g, at = _table(state, state["grad"])
        x, _ = _table(state, state["x"])
        gx = (g @ state["w"].float()).flatten(0, 1)[at]
        return {"grad_x": gx.to(_type(case["dtype"])),
                "grad_w": (g.transpose(1, 2) @ x).to(_type(case["out"]))}
    if op == "int8":
        q, s = _codes(state["x"])
        y = (q @ state["codes"].float().t()) * s * state["scales"]
        return {"out": y.to(_type(case["out"]))}
    if op == "silu":
        gate, up = state["a"].float().chunk(2, 1)
        return {"out": (gate / (1 + torch.exp(-gate)) * up).to(state["a"].dtype)}
    if op == "silu_grad":
        return {"grad": _silu_grad(state["grad"], state["a"]).to(state["a"].dtype)}
    if op == "gather":
        return {"rows": state["x"][state["row_src"].long() // case["k"]]}
    live = state["slot_dst"] >= 0
    at = state["slot_dst"].clamp(min=0).long()
    weights = state["weights"] * live
    if op == "combine":
        y = state["y"].float()[at.flatten()].view(*at.shape, -1)
        return {"out": (y * weights.unsqueeze(-1)).sum(1).to(state["y"].dtype)}
    grad = state["grad"].float()
    src = state["row_src"].long()
    gy = grad[src // case["k"]] * weights.flatten()[src].unsqueeze(1)
    gw = torch.stack([(state["y"].float()[at[:, j]] * grad).sum(1) for j in range(case["k"])], 1)
    return {"grad_y": gy.to(state["y"].dtype), "grad_weights": gw * live}


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def _own(state):
    from nvfp4_block_scaled_topk_gb300 import megamoe

    case = state["case"]
    op = case["op"]
    if op == "grouped":
        return {"out": megamoe.grouped_linear(state["x"], state["w"], state["offsets"],
                                              out_dtype=_type(case["out"]))}
    if op == "grouped_grad":
        gx, gw = megamoe.grouped_linear_backward(state["grad"], state["x"], state["w"],
                                                 state["offsets"],
                                                 grad_w_dtype=_type(case["out"]))
        return {"grad_x": gx, "grad_w": gw}
    if op == "int8":
        epi = megamoe.EPI_F32 if case["out"] == "float32" else megamoe.EPI_BF16
        return {"out": megamoe.linear_int8(state["x"], state["weight"], epi)[0]}
    if op == "silu":
        return {"out": megamoe.silu_mul(state["a"])}
    if op == "silu_grad":
        return {"grad": megamoe.silu_mul_backward(state["grad"], state["a"])}
    if op == "gather":
        return {"rows": megamoe.gather_rows(state["x"], state["row_src"], case["k"])}
    if op == "combine":
        return {"out": megamoe.combine_rows(state["y"], state["slot_dst"], state["weights"])}
    gy, gw = megamoe.combine_rows_backward(state["grad"], state["y"], state["slot_dst"],
                                           state["weights"])
    return {"grad_y": gy, "grad_weights": gw}


def run(state):
    return _own(state) if own else _plain(state)


def _bytes(name):
    return 4 if name == "float32" else 2


def work(case):
    """Bytes: inputs once (the weights of experts that have rows), outputs once.
    Operations: the products, or a handful for each element."""
    op = case["op"]
    if op in ("grouped", "grouped_grad"):
        T, E, k, K, N = (case[n] for n in ("T", "E", "k", "K", "N"))
        rows = T * k * (1 - case["dropped"])
        weights = E * (1 - (1 - k / E) ** T) * K * N if k < E else E * K * N
        size = _bytes(case["out"])
        if op == "grouped":
            return {"bytes": 2 * weights + rows * (2 * K + size * N), "flops": 2 * rows * K * N}
        return {"bytes": 2 * weights + size * E * K * N + rows * (4 * K + 2 * N),
                "flops": 4 * rows * K * N}
    if op == "int8":
        T, K, N = case["T"], case["K"], case["N"]
        return {"bytes": _bytes(case["dtype"]) * T * K + N * (K + 4) + _bytes(case["out"]) * T * N,
                "flops": 2 * T * K * N}
    if op in ("silu", "silu_grad"):
        n = case["rows"] * case["I"]
        return {"bytes": n * (6 if op == "silu" else 10), "flops": n * (6 if op == "silu" else 12)}
    T, slots, d = case["T"], case["T"] * case["k"], case["d"]
    rows = slots * (1 - case["dropped"])
    if op == "gather":
        return {"bytes": 2 * d * (T + rows) + 4 * rows, "flops": 0}
    if op == "combine":
        return {"bytes": 2 * d * (T + rows) + 8 * slots, "flops": 2 * rows * d}
    return {"bytes": 2 * d * (T + 2 * rows) + 12 * slots, "flops": 3 * rows * d}


# --------------------------------------------------------------------------
# the operators in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    op = case["op"]
    v = _inputs(case, seed)
    if op in ("grouped", "grouped_grad"):
        if work(case)["flops"] > 4e12:
            return None
        x, ends = v["x"].double(), v["offsets"].tolist()
        if op == "grouped":
            out = torch.empty((len(x), case["N"]), dtype=torch.float64, device="cuda")
            for e, (a, b) in enumerate(zip(ends, ends[1:])):
                out[a:b] = x[a:b] @ v["w"][e].double().t()
            return {"out": out}
        grad, gx, gw = v["grad"].double(), torch.empty_like(x), []
        for e, (a, b) in enumerate(zip(ends, ends[1:])):
            gx[a:b] = grad[a:b] @ v["w"][e].double()
            gw.append(grad[a:b].t() @ x[a:b])
        return {"grad_x": gx, "grad_w": torch.stack(gw)}
    if op == "int8":
        x = v["x"].double()
        scale = x.abs().max(1, keepdim=True)[0] / 127
        q = torch.round(x * 127 / (scale * 127).clamp(min=1e-300))
        return {"out": (q * scale) @ (v["codes"].double() * v["scales"].double().unsqueeze(1)).t()}
    if op in ("silu", "silu_grad"):
        a = v["a"].double()
        gate, up = a[:, :case["I"]], a[:, case["I"]:]
        s = torch.sigmoid(gate)
        if op == "silu":
            return {"out": gate * s * up}
        g = v["grad"].double()
        return {"grad": torch.cat([g * up * (s + gate * s * (1 - s)), g * gate * s], 1)}
    dst = v["slot_dst"].long()
    if op == "gather":
        rows = torch.empty((v["live"], case["d"]), dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            t = (dst[:, j] >= 0).nonzero().flatten()
            rows[dst[t, j]] = v["x"][t].double()
        return {"rows": rows}
    if op == "combine":
        out = torch.zeros((case["T"], case["d"]), dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            t = (dst[:, j] >= 0).nonzero().flatten()
            out[t] += v["y"][dst[t, j]].double() * v["weights"][t, j].double().unsqueeze(1)
        return {"out": out}
    gy = torch.empty((v["live"], case["d"]), dtype=torch.float64, device="cuda")
    gw = torch.zeros((case["T"], case["k"]), dtype=torch.float64, device="cuda")
    for j in range(case["k"]):
        t = (dst[:, j] >= 0).nonzero().flatten()
        g = v["grad"][t].double()
        gy[dst[t, j]] = g * v["weights"][t, j].double().unsqueeze(1)
        gw[t, j] = (g * v["y"][dst[t, j]].double()).sum(1)
    return {"grad_y": gy, "grad_weights": gw}
