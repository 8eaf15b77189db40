"""Products grouped by expert, their gradients, the gated activation and the
movement of rows against plain 64-bit forms.

Products: the factors of a product are exact in fp32; the tensor cores add K / 16
groups of them into an fp32 sum, each addition off by at most one unit of 2^-23 of
what has been added up so far: |got - want| <= (K / 16 + 2) 2^-23 sum |p q|, plus
half a step of the output type (eps / 2 of the value, or half of the smallest
subnormal).
"""

import pytest
import torch

from nvfp4_block_scaled_topk_gb300 import megamoe

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
BF, FP = torch.bfloat16, torch.float16


def half_step(want, dtype):
    f = torch.finfo(dtype)
    return want.abs() * (f.eps / 2) + f.smallest_normal * f.eps / 2


def check(got, want, bound):
    dtype = got.dtype
    got = got.double()
    assert got.shape == want.shape
    bad = (got - want).abs() > bound + half_step(want.abs() + bound, dtype)
    bad |= ~torch.isfinite(got)
    assert not bad.any(), ((got - want)[bad][:4], bound.expand_as(want)[bad][:4], bad.nonzero()[:4])


def layout(counts, pad):
    """offsets, padded_offsets (int32, CUDA) and the rows that experts' rows span."""
    c = torch.tensor(counts)
    off = torch.zeros(len(counts) + 1, dtype=torch.int64)
    off[1:] = c.cumsum(0)
    poff = torch.zeros_like(off)
    poff[1:] = ((c + pad - 1) // pad * pad).cumsum(0)
    return off.int().cuda(), poff.int().cuda(), int(poff[-1])


def strided(t, extra=8):
    """The same values in rows of a wider matrix."""
    return torch.cat([t, torch.full((t.shape[0], extra), 9.0, dtype=t.dtype, device=t.device)],
                     1)[:, :t.shape[1]]


def make(counts, K, N, dtype, pad=1, behind=5, seed=0):
    """x, grad, w, offsets, padded offsets, rows of each expert; padding rows and
    rows behind the last expert hold NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    off, poff, span = layout(counts, pad)
    rows = span + behind
    x = torch.full((rows, K), float("nan"), device="cuda")
    gr = torch.full((rows, N), float("nan"), device="cuda")
    where = []
    for e, c in enumerate(counts):
        s = int(poff[e])
        x[s:s + c] = torch.randn((c, K), generator=g, device="cuda")
        gr[s:s + c] = torch.randn((c, N), generator=g, device="cuda")
        where.append((s, c))
    w = torch.randn((len(counts), N, K), generator=g, device="cuda") / 8
    return x.to(dtype), gr.to(dtype), w.to(dtype), off, poff, where


SHAPES = [  # counts, K, N
    ([1], 64, 64), ([1], 8, 8), ([3, 0, 1], 72, 264), ([0, 17, 0, 300, 16, 0], 200, 136),
    ([257, 255, 256, 1], 64, 520), ([31, 33, 64, 65, 129], 1000, 72), ([600], 328, 256),
    ([0, 0, 5], 7168, 40), ([2] * 40 + [0, 90], 136, 1032), ([1] * 130, 64, 64)]


@pytest.mark.parametrize("counts,K,N", SHAPES)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("pad", [1, 32])
def test_forward(cuda_lib, counts, K, N, dtype, pad):
    x, _, w, off, poff, where = make(counts, K, N, dtype, pad)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for out_dtype in (dtype, torch.float32):
        wide = torch.full((x.shape[0], N + 8), 7.0, dtype=out_dtype, device="cuda")
        out = wide[:, :N]
        got = megamoe.grouped_linear(strided(x), w, off, poff, out_dtype=out_dtype, out=out,
                                     status=status)
        assert got is out and int(status) == 0
        owned = torch.zeros(x.shape[0], dtype=torch.bool, device="cuda")
        for e, (s, c) in enumerate(where):
            p, q = x[s:s + c].double(), w[e].double()
            check(out[s:s + c], p @ q.t(), (K / 16 + 2) * U * (p.abs() @ q.abs().t()))
            owned[s:s + c] = True
        assert (wide[~owned] == 7).all() and (wide[:, N:] == 7).all()
    if pad == 1:  # no padded offsets, contiguous rows
        again = megamoe.grouped_linear(x, w, off, out_dtype=torch.float32)
        assert torch.equal(again[owned], out[owned])


@pytest.mark.parametrize("counts,K,N", SHAPES)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("pad", [1, 32])
def test_backward(cuda_lib, counts, K, N, dtype, pad):
    x, grad, w, off, poff, where = make(counts, K, N, dtype, pad, seed=1)
    for w_dtype in (dtype, torch.float32):
        wide = torch.full((x.shape[0], K + 8), 7.0, dtype=dtype, device="cuda")
        gx, gw = megamoe.grouped_linear_backward(strided(grad), strided(x), w, off, poff,
                                                 grad_w_dtype=w_dtype, grad_x=wide[:, :K])
        assert gw.dtype == w_dtype
        owned = torch.zeros(x.shape[0], dtype=torch.bool, device="cuda")
        for e, (s, c) in enumerate(where):
            p, g, q = x[s:s + c].double(), grad[s:s + c].double(), w[e].double()
            check(gx[s:s + c], g @ q, (N / 16 + 2) * U * (g.abs() @ q.abs()))
            check(gw[e], g.t() @ p, (c / 16 + 2) * U * (g.abs().t() @ p.abs()))
            if c == 0:
                assert (gw[e] == 0).all()
            owned[s:s + c] = True
        assert (wide[~owned] == 7).all() and (wide[:, K:] == 7).all()
    one, none = megamoe.grouped_linear_backward(grad, x, w, off, poff, need_w=False)
    assert none is None and torch.equal(one[owned], gx[owned])
    none, one = megamoe.grouped_linear_backward(grad, x, w, off, poff, need_x=False)
    assert none is None and torch.equal(one, gw)


def test_experts_keep_to_themselves(cuda_lib):
    """Inf and NaN of one expert's rows and weights reach no other expert."""
    counts, K, N = [20, 33, 47], 136, 264
    x, grad, w, off, poff, where = make(counts, K, N, BF, seed=2)
    clean = (megamoe.grouped_linear(x, w, off), *megamoe.grouped_linear_backward(grad, x, w, off))
    for bad in (float("inf"), float("nan")):
        x2, g2, w2 = x.clone(), grad.clone(), w.clone()
        s, c = where[1]
        x2[s:s + c] = bad
        g2[s:s + c] = bad
        w2[1] = bad
        out = (megamoe.grouped_linear(x2, w2, off), *megamoe.grouped_linear_backward(g2, x2, w2, off))
        for e in (0, 2):
            a, b = where[e][0], where[e][0] + where[e][1]
            assert torch.equal(out[0][a:b], clean[0][a:b])
            assert torch.equal(out[1][a:b], clean[1][a:b])
            assert torch.equal(out[2][e], clean[2][e])
        assert not torch.isfinite(out[0][s:s + c]).any() and not torch.isfinite(out[2][1]).any()


def test_no_rows(cuda_lib):
    w = torch.randn((3, 16, 24), device="cuda").to(BF)
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    x, grad = torch.empty((0, 24), dtype=BF, device="cuda"), torch.empty((0, 16), dtype=BF, device="cuda")
    assert megamoe.grouped_linear(x, w, off).shape == (0, 16)
    gx, gw = megamoe.grouped_linear_backward(grad, x, w, off)
    assert gx.shape == (0, 24) and gw.shape == w.shape and (gw == 0).all()
    # rows, but none of any expert
    x, grad = torch.ones((5, 24), dtype=BF, device="cuda"), torch.ones((5, 16), dtype=BF, device="cuda")
    out = torch.full((5, 16), 3.0, dtype=BF, device="cuda")
    assert (megamoe.grouped_linear(x, w, off, out=out) == 3).all()
    assert (megamoe.grouped_linear_backward(grad, x, w, off)[1] == 0).all()


def test_offsets_outside_the_matrix(cuda_lib):
    """Rows outside are left out, and the status says so."""
    x, grad, w, off, _, where = make([4, 5, 6], 64, 72, BF, behind=0)
    for change in ([0, 4, 9, 400], [-7, 4, 9, 15], [0, 4, 2, 15], [100, 200, 300, 400]):
        bad = torch.tensor(change, dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((15, 72), 3.0, dtype=BF, device="cuda")
        megamoe.grouped_linear(x, w, bad, out=out, status=status)
        assert int(status) == megamoe.DEV_BAD_OFFSETS
        if change[1] == 4 and change[2] == 9:
            want = x[4:9].double() @ w[1].double().t()
            check(out[4:9], want, 6 * U * (x[4:9].double().abs() @ w[1].double().abs().t()))
        status.zero_()
        _, gw = megamoe.grouped_linear_backward(grad, x, w, bad, status=status)
        assert int(status) == megamoe.DEV_BAD_OFFSETS and torch.isfinite(gw).all()


@pytest.mark.parametrize("rows,I", [(1, 8), (3, 64), (48, 2048), (130, 264), (1000, 40)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_silu(cuda_lib, rows, I, dtype):
    """Off by a few units of fp32, |g| 2^-24 from the exponential's argument among
    them, and half a step."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    a = torch.randn((rows, 2 * I), generator=g, device="cuda") * 6
    a[0, :4] = torch.tensor([0.0, -100.0, 100.0, -17.0])
    a, grad = a.to(dtype), torch.randn((rows, I), generator=g, device="cuda").to(dtype)
    x = a.double()
    gate, up = x[:, :I], x[:, I:]
    s = torch.sigmoid(gate)
    rel = (gate.abs() + 12) * 2.0 ** -23
    tiny = 2.0 ** -120  # exponentials below the smallest normal are 0
    want = gate * s * up
    check(megamoe.silu_mul(strided(a)), want, rel * want.abs() + tiny)
    h = grad.double()
    dg, du = h * up * (s + gate * s * (1 - s)), h * gate * s
    # the two terms of 1 + g (1 - s) may cancel
    room = torch.cat([rel * (h * up * s).abs() * (1 + (gate * (1 - s)).abs()), rel * du.abs()], 1)
    got = megamoe.silu_mul_backward(strided(grad), strided(a))
    check(got, torch.cat([dg, du], 1), room + tiny)
    # differences of the 64-bit form
    d = 1e-5
    f = lambda p, q: p * torch.sigmoid(p) * q  # noqa: E731
    assert torch.allclose(dg, h * (f(gate + d, up) - f(gate - d, up)) / (2 * d), rtol=1e-5, atol=1e-6)
    assert torch.allclose(du, h * (f(gate, up + d) - f(gate, up - d)) / (2 * d), rtol=1e-5, atol=1e-6)
    # rows from live_rows on are left as they are
    for live in (0, rows // 2, rows, rows + 7):
        n = torch.tensor([live], dtype=torch.int32, device="cuda")
        out = torch.full((rows, I), 5.0, dtype=dtype, device="cuda")
        ga = torch.full((rows, 2 * I), 5.0, dtype=dtype, device="cuda")
        megamoe.silu_mul(a, live_rows=n, out=out)
        megamoe.silu_mul_backward(grad, a, live_rows=n, grad_a=ga)
        assert (out[live:] == 5).all() and (ga[live:] == 5).all()
        assert torch.equal(ga[:live], got[:live])


def routed(T, k, E, dropped=0.1, seed=0):
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand((T, E), generator=g).argsort(1)[:, :k].to(torch.int32)
    ids[torch.rand((T, k), generator=g) < dropped] = -1
    return ids.cuda()


@pytest.mark.parametrize("T,k,E,d", [(1, 1, 1, 8), (1, 6, 48, 7168), (33, 3, 5, 264), (257, 16, 16, 40),
                                     (130, 8, 12, 2056)])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("pad", [1, 32])
def test_rows(cuda_lib, T, k, E, d, dtype, pad):
    g = torch.Generator(device="cuda").manual_seed(T + k)
    ids = routed(T, k, E, dropped=0.1 if T > 1 else 0)
    r = megamoe.route_permute(ids, E, pad)
    src, dst = r["row_src"], r["slot_dst"].view(T, k)
    rows = src.numel()
    x = torch.randn((T, d), generator=g, device="cuda").to(dtype)
    w = torch.rand((T, k), generator=g, device="cuda")
    got = megamoe.gather_rows(strided(x), src, k)
    taken = src >= 0
    assert torch.equal(got[taken], x[src[taken].long() // k]) and (got[~taken] == 0).all()

    y = torch.randn((rows, d), generator=g, device="cuda").to(dtype)
    y[~taken] = float("nan")
    live = (dst >= 0).unsqueeze(-1)
    picked = torch.where(live, y[dst.clamp(min=0).long()].double(), 0.0)
    for weights in (w, None):
        f = torch.ones_like(w) if weights is None else weights
        terms = picked * f.double().unsqueeze(-1)
        # k products and sums, each rounded to fp32
        check(megamoe.combine_rows(strided(y), dst, weights), terms.sum(1),
              2 * k * 2.0 ** -24 * terms.abs().sum(1))
        go = torch.randn((T, d), generator=g, device="cuda").to(dtype)
        gy = torch.full((rows, d), 5.0, dtype=dtype, device="cuda")
        _, gw = megamoe.combine_rows_backward(strided(go), strided(y), dst, weights, grad_y=gy)
        want = go[src[taken].long() // k].double() * f.flatten()[src[taken].long()].double().unsqueeze(1)
        check(gy[taken], want, 2.0 ** -24 * want.abs())
        assert (gy[~taken] == 5).all()
        dots = picked * go.double().unsqueeze(1)
        # a lane's sums of its elements, then 5 + 8 more
        check(gw, dots.sum(-1), (d / 16 + 40) * 2.0 ** -24 * dots.abs().sum(-1))
        assert (gw[dst < 0] == 0).all()
        assert megamoe.combine_rows_backward(go, y, dst, weights, need_weights=False)[1] is None
    # the gradient of gather_rows
    gr = torch.randn((rows, d), generator=g, device="cuda").to(dtype)
    want = torch.where(live, gr[dst.clamp(min=0).long()].double(), 0.0)
    check(megamoe.combine_rows(gr, dst), want.sum(1), 2 * k * 2.0 ** -24 * want.abs().sum(1))


def test_rows_outside(cuda_lib):
    """Indices past the matrices count as none."""
    x = torch.randn((3, 16), device="cuda").to(BF)
    src = torch.tensor([0, 5, 6, 700, -1], dtype=torch.int32, device="cuda")
    got = megamoe.gather_rows(x, src, 2)
    assert torch.equal(got[:2], x[[0, 2]]) and (got[2:] == 0).all()
    dst = torch.tensor([[0, 3], [9, 1], [-4, 1 << 30]], dtype=torch.int32, device="cuda")
    out = megamoe.combine_rows(x, dst)
    assert torch.equal(out[:2], x[[0, 1]]) and (out[2] == 0).all()
    gy, gw = megamoe.combine_rows_backward(x, x, dst, grad_y=torch.zeros_like(x))
    assert torch.equal(gy[:2], x[:2]) and (gy[2] == 0).all()
    assert (gw[2] == 0).all() and gw[0, 1] == 0 and gw[1, 0] == 0


def test_layer_and_gradients(cuda_lib):
    """Route, gather, gate and up, activation, down, combine; and back.  Each step of the
    64-bit form starts from the values that the step before gave, so that each is held
    to its own roundings."""
    T, k, E, d, I = 100, 3, 7, 264, 136
    g = torch.Generator(device="cuda").manual_seed(11)
    x = torch.randn((T, d), generator=g, device="cuda").to(BF)
    w13 = (torch.randn((E, 2 * I, d), generator=g, device="cuda") / 16).to(BF)
    w2 = (torch.randn((E, d, I), generator=g, device="cuda") / 16).to(BF)
    logits = torch.randn((T, E), generator=g, device="cuda")
    go = torch.randn((T, d), generator=g, device="cuda").to(BF)

    ids, tw = megamoe.router_scored_topk(logits, k)
    r = megamoe.route_permute(ids, E)
    off, dst, live = r["offsets"], r["slot_dst"].view(T, k), r["offsets"][E:]
    xr = megamoe.gather_rows(x, r["row_src"], k)
    a = megamoe.grouped_linear(xr, w13, off)
    h = megamoe.silu_mul(a, live_rows=live)
    y = megamoe.grouped_linear(h, w2, off)
    out = megamoe.combine_rows(y, dst, tw)
    gy, gtw = megamoe.combine_rows_backward(go, y, dst, tw)
    gh, gw2 = megamoe.grouped_linear_backward(gy, h, w2, off)
    ga = megamoe.silu_mul_backward(gh, a, live_rows=live)
    gxr, gw13 = megamoe.grouped_linear_backward(ga, xr, w13, off)
    gx = megamoe.combine_rows(gxr, dst)
    glogits = megamoe.router_scored_topk_backward(logits, ids, gtw)

    # the whole in 64 bits from the inputs, by automatic differentiation
    leaves = [t.double().requires_grad_() for t in (x, w13, w2, logits)]
    X, W13, W2, L = leaves
    s = torch.sigmoid(L).gather(1, ids.long())
    TW = s / s.sum(1, keepdim=True)
    Y = []
    for j in range(k):
        e = ids[:, j].long()
        A = torch.einsum("td,tnd->tn", X, W13[e])
        H = A[:, :I] * torch.sigmoid(A[:, :I]) * A[:, I:]
        Y.append(torch.einsum("ti,tdi->td", H, W2[e]) * TW[:, j:j + 1])
    OUT = torch.stack(Y).sum(0)
    OUT.backward(go.double())
    # every bf16 intermediate is off by 2^-8 of itself at most (half a step); six of
    # them lie between an input and the furthest gradient: six such shares of the norm
    # bound the whole's
    for got, want in ((out, OUT), (gx, X.grad), (gw13, W13.grad), (gw2, W2.grad), (glogits, L.grad)):
        want = want.detach()
        rel = (got.double() - want).norm() / want.norm()
        assert rel < 6 * 2.0 ** -8, rel
