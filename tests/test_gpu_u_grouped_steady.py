"""The 16-bit experts' operators and the integer linear over and over: more tiles than
CTAs and more steps than stages, graphs, other streams, waits that run out, rows whose
offsets pass 32 bits, and tensors that the binding refuses."""

import pytest
import torch

from nvfp4_block_scaled_topk_gb300 import megamoe

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
U = 2.0 ** -23


def _counts(E, most, seed):
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(0, most, (E,), generator=g)
    c[E // 2] = 0
    off = torch.zeros(E + 1, dtype=torch.int64)
    off[1:] = c.cumsum(0)
    return off


def _case(E, most, K, N, seed=0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    off = _counts(E, most, seed)
    R = int(off[-1])
    x = torch.randn((R, K), generator=g, device="cuda").to(dtype)
    gr = torch.randn((R, N), generator=g, device="cuda").to(dtype)
    w = (torch.randn((E, N, K), generator=g, device="cuda") / 16).to(dtype)
    return x, gr, w, off


def _within(got, want, bound):
    f = torch.finfo(got.dtype)
    err = (got.double() - want).abs()
    assert (err <= bound + (want.abs() + bound) * f.eps / 2 + f.smallest_normal * f.eps).all()


@pytest.mark.parametrize("E,most,K,N", [(24, 700, 1160, 1544), (150, 70, 520, 776)])
@pytest.mark.parametrize("out", [BF, torch.float32])
def test_many_tiles(cuda_lib, E, most, K, N, out):
    x, gr, w, off = _case(E, most, K, N)
    dev = off.int().cuda()
    y = megamoe.grouped_linear(x, w, dev, out_dtype=out)
    gx, gw = megamoe.grouped_linear_backward(gr, x, w, dev, grad_w_dtype=out)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        p, q, g = x[a:b].double(), w[e].double(), gr[a:b].double()
        _within(y[a:b], p @ q.t(), (K / 16 + 2) * U * (p.abs() @ q.abs().t()))
        _within(gx[a:b], g @ q, (N / 16 + 2) * U * (g.abs() @ q.abs()))
        _within(gw[e], g.t() @ p, ((b - a) / 16 + 2) * U * (g.abs().t() @ p.abs()))


def test_long_sums_keep_their_last_bits(cuda_lib):
    """fp32 results of sums of 16384: parts of 512 terms, each off by at most one unit of
    2^-24 for each of its 32 additions of what it has added up, then rounded sums."""
    R, K, N = 16384, 136, 264
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((R, K), generator=g, device="cuda").to(BF)
    gr = torch.randn((R, N), generator=g, device="cuda").to(BF)
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    _, gw = megamoe.grouped_linear_backward(gr, x, torch.zeros((1, N, K), device="cuda").to(BF), off,
                                            need_x=False)
    want = gr.double().t() @ x.double()
    # a part of 512 normal products is about sqrt(512), its error at most 32 units of it;
    # 32 independent parts: the same share of their sum
    assert ((gw[0].double() - want).norm() / want.norm()) < 32 * 2.0 ** -23
    w = torch.randn((1, N, R), generator=g, device="cuda").to(BF)
    t = torch.randn((48, R), generator=g, device="cuda").to(BF)
    one = torch.tensor([0, 48], dtype=torch.int32, device="cuda")
    y = megamoe.grouped_linear(t, w, one, out_dtype=torch.float32)
    want = t.double() @ w[0].double().t()
    assert ((y.double() - want).norm() / want.norm()) < 32 * 2.0 ** -23


@pytest.mark.parametrize("T,K,N", [(2, 1536, 2048), (11, 1536, 2048), (70, 2064, 520), (1500, 1040, 4104)])
def test_int8_many(cuda_lib, T, K, N):
    g = torch.Generator().manual_seed(T)
    q = torch.randint(-40, 41, (T, K), generator=g, dtype=torch.int8).cuda()
    w = torch.randint(-40, 41, (N, K), generator=g, dtype=torch.int8).cuda()
    one, sx = torch.ones(N, device="cuda"), torch.ones(T, device="cuda")
    weight = megamoe.Int8LinearWeights(N, K, w, one)
    want = (q.double() @ w.double().t()).float()
    ws = None
    for _ in range(3):
        got, ws = megamoe.linear_int8(q, weight, megamoe.EPI_F32, x_scales=sx, ws=ws)
        assert torch.equal(got, want)


def _all(x, gr, w, off, ids, tw, weight):
    """Every operator once, on the current stream."""
    E = w.shape[0]
    r = megamoe.route_permute(ids, E)
    rows = megamoe.gather_rows(x, r["row_src"], ids.shape[1])
    y = megamoe.grouped_linear(rows, w, r["offsets"])
    h = megamoe.silu_mul(y, live_rows=r["offsets"][E:])
    out = megamoe.combine_rows(y, r["slot_dst"].view(ids.shape), tw)
    gy, gw = megamoe.combine_rows_backward(out, y, r["slot_dst"].view(ids.shape), tw)
    gx, gww = megamoe.grouped_linear_backward(gy, rows, w, r["offsets"])
    ga = megamoe.silu_mul_backward(h, y, live_rows=r["offsets"][E:])
    i8 = [megamoe.linear_int8(x[:n], weight)[0] for n in (1, 9, len(x))]
    return [out, gy, gw, gx, gww, h, ga, *i8]


def _inputs(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, k, E, d, N = 90, 3, 6, 256, 528
    x = torch.randn((T, d), generator=g, device="cuda").to(BF)
    w = (torch.randn((E, N, d), generator=g, device="cuda") / 16).to(BF)
    ids = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous()
    tw = torch.rand((T, k), generator=g, device="cuda")
    master = torch.randn((N, d), generator=g, device="cuda")
    return x, None, w, None, ids, tw, master


def test_graphs_and_streams(cuda_lib):
    """Two captured graphs replayed with new inputs, and calls on other streams at once:
    the same bits as one call after another."""
    sets = [_inputs(s) for s in range(3)]
    want = [[t.clone() for t in _all(*s[:-1], megamoe.Int8LinearWeights.quantize(s[-1]))] for s in sets]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        held = [t.clone() if t is not None else None for t in sets[0]]
        weight = megamoe.Int8LinearWeights.quantize(held[-1])
        _all(*held[:-1], weight)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            codes, scales = megamoe.quantize_int8(held[-1])
            weight.codes.copy_(codes)
            weight.scales.copy_(scales)
            got = _all(*held[:-1], weight)
        graphs.append((graph, held, got))
    for turn in (1, 2, 0):
        for graph, held, got in graphs:
            for t, s in zip(held, sets[turn]):
                if t is not None:
                    t.copy_(s)
            graph.replay()
        torch.cuda.synchronize()
        for _, _, got in graphs:
            for a, b in zip(got, want[turn]):
                assert torch.equal(a, b)
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for s, st in zip(sets, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(_all(*s[:-1], megamoe.Int8LinearWeights.quantize(s[-1])))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


# one stage and more than the ring holds, rows that end inside a stage, both outputs
@pytest.mark.parametrize("most,K,N", [(40, 64, 72), (300, 1096, 520)])
@pytest.mark.parametrize("out", [BF, torch.float32])
def test_waits_that_run_out(cuda_lib, most, K, N, out):
    x, gr, w, off = _case(20, most, K, N, seed=3)
    off = off.int().cuda()

    def calls(status):
        return (megamoe.grouped_linear(x, w, off, out_dtype=out, status=status),
                *megamoe.grouped_linear_backward(gr, x, w, off, grad_w_dtype=out, status=status))

    want = calls(None)
    torch.cuda.synchronize()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    megamoe.set_wait_limit_ns(100)
    try:
        calls(status)
        torch.cuda.synchronize()
        assert int(status) == megamoe.DEV_TIMEOUT
    finally:
        megamoe.set_wait_limit_ns(0)
    status.zero_()
    for a, b in zip(calls(status), want):
        assert torch.equal(a, b)
    assert int(status) == 0


@pytest.mark.parametrize("T,K,N", [(17, 128, 72), (300, 4112, 520)])
def test_int8_waits_that_run_out(cuda_lib, T, K, N):
    x = torch.randn((T, K), device="cuda").to(BF)
    weight = megamoe.Int8LinearWeights.quantize(torch.randn((N, K), device="cuda"))
    want, ws = megamoe.linear_int8(x, weight)
    torch.cuda.synchronize()
    megamoe.set_wait_limit_ns(100)
    try:
        megamoe.linear_int8(x, weight, ws=ws)
        torch.cuda.synchronize()
        assert int(ws[:4].view(torch.int32)) == megamoe.DEV_TIMEOUT
    finally:
        megamoe.set_wait_limit_ns(0)
    got, _ = megamoe.linear_int8(x, weight, ws=ws)
    assert torch.equal(got, want) and int(ws[:4].view(torch.int32)) == 0


def _wide(t, ld):
    """The same rows `ld` elements apart, most of the memory between them untouched."""
    far = torch.empty_strided(t.shape, (ld, 1), dtype=t.dtype, device=t.device)
    far.copy_(t)
    return far


def test_rows_far_apart(cuda_lib):
    """Offsets past 2^32 elements."""
    ld = 1 << 28
    g = torch.Generator(device="cuda").manual_seed(1)
    R, K, N, k = 20, 72, 136, 2
    x = torch.randn((R, K), generator=g, device="cuda").to(BF)
    gr = torch.randn((R, N), generator=g, device="cuda").to(BF)
    w = torch.randn((3, N, K), generator=g, device="cuda").to(BF)
    off = torch.tensor([0, 9, 9, 20], dtype=torch.int32, device="cuda")
    y = megamoe.grouped_linear(x, w, off)
    gx, gw = megamoe.grouped_linear_backward(gr, x, w, off)
    out = _wide(torch.zeros_like(gr), ld)
    assert torch.equal(megamoe.grouped_linear(_wide(x, ld), w, off, out=out), y)
    del out
    far = megamoe.grouped_linear_backward(_wide(gr, ld), x, w, off, grad_x=_wide(x, ld))
    assert torch.equal(far[0], gx) and torch.equal(far[1], gw)
    del far
    # (half of 136 is no multiple of 8: the first 128 columns)
    assert torch.equal(megamoe.silu_mul(_wide(gr, ld)[:, :128]), megamoe.silu_mul(gr[:, :128]))
    src = torch.arange(R - 1, -1, -1, dtype=torch.int32, device="cuda")
    rows = megamoe.gather_rows(_wide(x, ld), src, 1)
    assert torch.equal(rows, x.flip(0))
    dst = src.view(R // k, k)
    assert torch.equal(megamoe.combine_rows(_wide(gr, ld), dst), megamoe.combine_rows(gr, dst))
    go = torch.randn((R // k, N), generator=g, device="cuda").to(BF)
    far = megamoe.combine_rows_backward(_wide(go, ld), _wide(gr, ld), dst, grad_y=_wide(gr, ld))
    near = megamoe.combine_rows_backward(go, gr, dst)
    assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])
    del far
    weight = megamoe.Int8LinearWeights.quantize(torch.randn((40, 128), device="cuda"))
    for T in (3, 10, 20):
        t = torch.randn((T, 128), generator=g, device="cuda").to(BF)
        want = megamoe.linear_int8(t, weight)[0]
        out = _wide(torch.zeros_like(want), ld)
        assert torch.equal(megamoe.linear_int8(_wide(t, ld), weight, out=out)[0], want)
        del out


def test_refusals(cuda_lib):
    x = torch.ones((6, 64), device="cuda").to(BF)
    w = torch.ones((2, 72, 64), device="cuda").to(BF)
    g = torch.ones((6, 72), device="cuda").to(BF)
    off = torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda")
    grouped, back = megamoe.grouped_linear, megamoe.grouped_linear_backward
    for error, call in [
            (TypeError, lambda: grouped(x.float(), w, off)), (TypeError, lambda: grouped(x, w.half(), off)),
            (TypeError, lambda: grouped(x, w.transpose(1, 2), off)), (TypeError, lambda: grouped(x, w[0], off)),
            (TypeError, lambda: grouped(x.t(), w, off)), (TypeError, lambda: grouped(x, w, off.long())),
            (TypeError, lambda: grouped(x, w, off.cpu())), (ValueError, lambda: grouped(x, w, off[:2])),
            (ValueError, lambda: grouped(x[:, :32], w, off)), (ValueError, lambda: grouped(x, w, off, off[:2])),
            (TypeError, lambda: grouped(x, w, off, out_dtype=torch.float16)),
            (ValueError, lambda: grouped(x, w, off, out=g[:3])), (TypeError, lambda: grouped(x, w, off, out=g.half())),
            (TypeError, lambda: grouped(x, w, off, status=torch.zeros(1, device="cuda"))),
            (megamoe.MegaMoEError, lambda: grouped(x[:, 1:], torch.ones((2, 72, 63), device="cuda").to(BF), off)),
            (ValueError, lambda: back(g[:5], x, w, off)), (TypeError, lambda: back(g.half(), x, w, off)),
            (ValueError, lambda: back(x, x, w, off)), (TypeError, lambda: back(g, x, w, off, grad_w_dtype=torch.float16)),
            (ValueError, lambda: back(g, x, w, off, grad_x=g)),
            (ValueError, lambda: megamoe.silu_mul(x[:, :63])), (TypeError, lambda: megamoe.silu_mul(x.double())),
            (ValueError, lambda: megamoe.silu_mul(x, live_rows=off)),
            (ValueError, lambda: megamoe.silu_mul_backward(x, x)),
            (TypeError, lambda: megamoe.silu_mul_backward(x[:, :32].half(), x)),
            (TypeError, lambda: megamoe.gather_rows(x, off.float(), 2)),
            (megamoe.MegaMoEError, lambda: megamoe.gather_rows(x, off, 0)),
            (ValueError, lambda: megamoe.combine_rows(x, off)),
            (ValueError, lambda: megamoe.combine_rows(x, off.view(3, 1), torch.ones(3, device="cuda"))),
            (TypeError, lambda: megamoe.combine_rows(x, off.view(3, 1), torch.ones((3, 1), device="cuda").half())),
            (ValueError, lambda: megamoe.combine_rows_backward(x, x, off.view(3, 1))),
            (TypeError, lambda: megamoe.quantize_int8(x.to(torch.int8))),
            (megamoe.MegaMoEError, lambda: megamoe.quantize_int8(x[:, :56]))]:
        with pytest.raises(error):
            call()
    weight = megamoe.Int8LinearWeights.quantize(w[0])
    codes = x.to(torch.int8)
    for error, call in [
            (TypeError, lambda: megamoe.linear_int8(codes, weight)),
            (TypeError, lambda: megamoe.linear_int8(x, weight, x_scales=torch.ones(6, device="cuda"))),
            (ValueError, lambda: megamoe.linear_int8(codes, weight, x_scales=torch.ones(5, device="cuda"))),
            (ValueError, lambda: megamoe.linear_int8(x[:, :48], weight)),
            (ValueError, lambda: megamoe.linear_int8(x, weight, out=g[:5])),
            (TypeError, lambda: megamoe.linear_int8(x, weight, ws=torch.zeros(4096, dtype=torch.uint8))),
            (megamoe.MegaMoEError, lambda: megamoe.linear_int8(
                x, weight, ws=torch.zeros(256, dtype=torch.uint8, device="cuda")))]:
        with pytest.raises(error):
            call()
    for n, k, c, s in ((72, 64, weight.codes.float(), weight.scales), (72, 64, weight.codes, weight.scales.cpu())):
        with pytest.raises(TypeError):
            megamoe.Int8LinearWeights(n, k, c, s)
    with pytest.raises(ValueError):
        megamoe.Int8LinearWeights(72, 48, weight.codes, weight.scales)


def test_one_row_of_any_stride(cuda_lib):
    x = torch.randn(1, 72, device="cuda").to(BF)
    odd = x.as_strided((1, 64), (65, 1))
    flat = odd.clone(memory_format=torch.contiguous_format)
    w = torch.randn((1, 40, 64), device="cuda").to(BF)
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    assert torch.equal(megamoe.grouped_linear(odd, w, off), megamoe.grouped_linear(flat, w, off))
    weight = megamoe.Int8LinearWeights.quantize(w[0])
    assert torch.equal(megamoe.linear_int8(odd, weight)[0], megamoe.linear_int8(flat, weight)[0])
    assert torch.equal(megamoe.silu_mul(odd), megamoe.silu_mul(flat))


def test_as_many_experts_as_there_may_be(cuda_lib):
    x, gr, w, off = _case(1024, 4, 64, 72, seed=6)
    dev = off.int().cuda()
    y = megamoe.grouped_linear(x, w, dev, out_dtype=torch.float32)
    gx, gw = megamoe.grouped_linear_backward(gr, x, w, dev)
    e = torch.repeat_interleave(torch.arange(1024), off[1:] - off[:-1]).cuda()
    p, q, g = x.double(), w.double()[e], gr.double()
    _within(y, torch.einsum("rk,rnk->rn", p, q), 6 * U * torch.einsum("rk,rnk->rn", p.abs(), q.abs()))
    _within(gx, torch.einsum("rn,rnk->rk", g, q), 7 * U * torch.einsum("rn,rnk->rk", g.abs(), q.abs()))
    outer = g.unsqueeze(2) * p.unsqueeze(1)
    want = torch.zeros((1024, 72, 64), dtype=torch.float64, device="cuda").index_add_(0, e, outer)
    most = torch.zeros_like(want).index_add_(0, e, outer.abs())
    _within(gw, want, 3 * U * most)


@pytest.mark.parametrize("dtype", [BF, torch.float16])
def test_ends_of_the_types(cuda_lib, dtype):
    """Subnormal and the largest operands, one product a sum: exact before the rounding."""
    f = torch.finfo(dtype)
    tiny = f.smallest_normal * f.eps
    a = torch.tensor([tiny, 3 * tiny, f.smallest_normal, 1.0, f.max, -tiny, 0.5, -f.max],
                     dtype=torch.float64)
    K = N = 64
    x = torch.zeros((len(a), K), dtype=torch.float64)
    x[torch.arange(len(a)), torch.arange(len(a))] = a
    w = torch.zeros((1, N, K), dtype=torch.float64)
    for i, v in enumerate(a):
        w[0, i] = v  # row i of w: the same value everywhere
    x, w = x.to(dtype).cuda(), w.to(dtype).cuda()
    off = torch.tensor([0, len(a)], dtype=torch.int32, device="cuda")
    want = (x.double() @ w[0].double().t()).float()  # products of two are exact in 64 bits
    got = megamoe.grouped_linear(x, w, off, out_dtype=torch.float32)
    # fp32's own subnormals may be lost: below 2^-126
    assert ((got == want) | ((want.abs() < 2.0 ** -126) & (got.abs() < 2.0 ** -126))).all()


# few tiles, whose sums two, three or four pairs of CTAs share; rows that end inside a
# part, a share of a row or none for some of them, an expert without rows
@pytest.mark.parametrize("counts", [[1], [0, 7, 0], [200], [30, 0, 3]])
@pytest.mark.parametrize("K,N", [(2056, 1032), (2120, 2600), (1544, 5000), (4104, 8200)])
@pytest.mark.parametrize("out", [torch.float16, torch.float32])
def test_shared_sums(cuda_lib, counts, K, N, out):
    g = torch.Generator(device="cuda").manual_seed(N)
    c = torch.tensor(counts)
    off = torch.cat([torch.zeros(1, dtype=torch.int64), c.cumsum(0)])
    R = int(off[-1])
    x = torch.randn((R + 2, K), generator=g, device="cuda").half()
    x[R:] = float("nan")
    w = (torch.randn((len(counts), N, K), generator=g, device="cuda") / 16).half()
    gr = torch.randn((R + 2, K), generator=g, device="cuda").half()
    gr[R:] = float("inf")
    wt = w.transpose(1, 2).contiguous()  # [E, K, N]: grad_x of it is a product with w
    dev = off.int().cuda()
    y = torch.full((R + 2, N), 7.0, dtype=out, device="cuda")
    megamoe.grouped_linear(x, w, dev, out_dtype=out, out=y)
    gx = torch.full((R + 2, N), 7.0, dtype=torch.float16, device="cuda")
    xn = torch.zeros((R + 2, N), dtype=torch.float16, device="cuda")
    megamoe.grouped_linear_backward(gr, xn, wt, dev, need_w=False, grad_x=gx)
    for e in range(len(counts)):
        a, b = int(off[e]), int(off[e + 1])
        q = w[e].double()
        for got, p in ((y, x[a:b].double()), (gx, gr[a:b].double())):
            _within(got[a:b], p @ q.t(), (K / 16 + 6) * U * (p.abs() @ q.abs().t()))
    assert (y[R:] == 7).all() and (gx[R:] == 7).all()
    again = megamoe.grouped_linear(x, w, dev, out_dtype=out)
    assert torch.equal(again[:R], y[:R])


@pytest.mark.parametrize("out", [BF, torch.float32])
def test_shared_waits_that_run_out(cuda_lib, out):
    x = torch.randn((8, 7168), device="cuda").to(BF)
    w = torch.randn((1, 2048, 7168), device="cuda").to(BF)
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    want = megamoe.grouped_linear(x, w, off, out_dtype=out)
    torch.cuda.synchronize()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    megamoe.set_wait_limit_ns(100)
    try:
        megamoe.grouped_linear(x, w, off, out_dtype=out, status=status)
        torch.cuda.synchronize()
        assert int(status) == megamoe.DEV_TIMEOUT
    finally:
        megamoe.set_wait_limit_ns(0)
    status.zero_()
    assert torch.equal(megamoe.grouped_linear(x, w, off, out_dtype=out, status=status), want)
    assert int(status) == 0


def test_an_expert_twice(cuda_lib):
    """A token that goes to one expert twice has two rows there."""
    ids = torch.tensor([[1, 1, 0], [2, 2, 2], [0, -1, 0]], dtype=torch.int32, device="cuda")
    x = torch.randn((3, 64), device="cuda").to(BF)
    tw = torch.rand((3, 3), device="cuda")
    r = megamoe.route_permute(ids, 3)
    dst = r["slot_dst"].view(3, 3)
    rows = megamoe.gather_rows(x, r["row_src"], 3)
    out = megamoe.combine_rows(rows, dst, tw)
    share = torch.where(ids >= 0, tw, 0.0).sum(1, keepdim=True).double()
    _within(out, x.double() * share, 4 * 2.0 ** -24 * x.double().abs() * 3)
    gy, gtw = megamoe.combine_rows_backward(x, rows, dst, tw)
    for t in range(3):
        for j in range(3):
            if ids[t, j] >= 0:
                _within(gy[dst[t, j]], x[t].double() * tw[t, j].double(), x[t].double().abs() * 2.0 ** -24)
    dots = (x.double() ** 2).sum(1, keepdim=True).expand(3, 3)
    _within(gtw, torch.where(ids >= 0, dots, 0.0), 44 * 2.0 ** -24 * dots)
    # one row in two slots: counted twice
    twice = torch.tensor([[0, 0]], dtype=torch.int32, device="cuda")
    assert torch.equal(megamoe.combine_rows(x, twice), 2 * x[:1])


@pytest.mark.parametrize("T", [3, 12, 70])
def test_graphs_that_share_a_workspace(cuda_lib, T):
    """Replayed one after the other; the status word is each call's own."""
    w = [megamoe.Int8LinearWeights.quantize(torch.randn((520, 2064), device="cuda")) for _ in range(2)]
    x = [torch.randn((T, 2064), device="cuda").to(BF) for _ in range(2)]
    want = [megamoe.linear_int8(a, b)[0] for a, b in zip(x, w)]
    ws = torch.empty(megamoe.linear_int8_workspace_size(T, 2064, 520) + 256, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for a, b in zip(x, w):
        megamoe.linear_int8(a, b, ws=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(megamoe.linear_int8(a, b, ws=ws)[0])
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    x[0][0, 5] = float("nan")
    graphs[0].replay()
    assert int(ws[:4].view(torch.int32)) == megamoe.DEV_NONFINITE
    graphs[1].replay()
    assert int(ws[:4].view(torch.int32)) == 0 and torch.equal(outs[1], want[1])
