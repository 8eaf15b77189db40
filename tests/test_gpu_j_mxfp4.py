"""MXFP4 quantisation, linear (and gradients) and routed experts against the
float64 oracle.

Codes, scales and values are exact.  A product's operands are the same values
on both sides and its terms are exact in fp32; the tensor cores add K / 64
groups of them into an fp32 sum, each addition off by at most one unit of
2^-23 of what has been added up so far, and splitting K adds at most 16 more:
|got - want| <= (K / 64 + 18) 2^-23 sum_k |p q|, plus half a unit of the output
type."""

import numpy as np
import pytest
import torch

from oracle import mxfp4 as mx
from nvfp4_block_scaled_topk_gb300 import megamoe
from helpers import assert_close_bf16, bf16_half_ulp

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


def _x(rows, K, dtype=torch.bfloat16, seed=0, wide=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=g)
    if wide:  # block magnitudes from 2^-12 to 2^6, and a block of zeros
        e = torch.randint(-12, 7, (rows, K // 32), generator=g).float()
        x = x * torch.exp2(e).repeat_interleave(32, 1)
        x[rows // 2, :32] = 0
    return x.to(dtype)


def _np(t):
    return t.double().cpu().numpy()


def _check_product(got, p, q, what):
    want = p @ q.T
    got = _np(got)
    bound = (p.shape[1] / 64 + 18) * U * (np.abs(p) @ np.abs(q).T) + 1e-38
    if what == torch.bfloat16:
        bound = bound + bf16_half_ulp(np.abs(want) + bound)
    assert got.shape == want.shape
    err = np.abs(got - want)
    assert (err <= bound).all(), (err - bound).max()


@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (130, 256), (31, 1536), (257, 480), (8, 7168)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_quantise_exact(cuda_lib, rows, K, dtype):
    x = _x(rows, K, dtype, seed=rows + K)
    for strided in (False, True):
        xs = x.cuda()
        if strided:
            xs = torch.cat([xs, torch.full((rows, 8), 7.0, dtype=dtype, device="cuda")], 1)[:, :K]
        for transpose in (False, True):
            ref = _np(x).T if transpose else _np(x)
            ref = np.pad(ref, ((0, 0), (0, -ref.shape[1] % 32)))
            code, byte = mx.encode(ref)
            codes, scales = megamoe.quantize_mxfp4(xs, transpose=transpose)
            assert np.array_equal(codes.cpu().numpy(), mx.pack(code))
            assert np.array_equal(scales.cpu().numpy(), byte)
            for dt in (torch.bfloat16, torch.float32):
                v = megamoe.dequantize_mxfp4(codes, scales, dtype=dt)
                assert v.dtype == dt and np.array_equal(_np(v), mx.decode(code, byte))
            _, at = megamoe.quantize_mxfp4(xs, transpose=transpose,
                                           scale_layout=megamoe.SCALES_MMA)
            want = mx.atoms(byte)
            at = at.cpu().numpy()
            r = ref.shape[0]
            # rows past the matrix are left as they are; compare its own
            real = mx.atoms(np.ones((r, -(-byte.shape[1] // 8) * 8), np.uint8)).astype(bool)
            assert np.array_equal(at[real], want[real])
            assert np.array_equal(megamoe.swizzle_scales_mxfp4(scales).cpu().numpy(), want)


def test_quantise_corners(cuda_lib):
    x = torch.zeros(8, 64)
    x[0, 0] = 2.0 ** -130          # a scale below the smallest: 2^-127
    x[1, 0] = float(np.finfo(np.float32).max)
    x[2, 5], x[2, 40] = torch.inf, 1.0
    x[3, 50] = torch.nan
    x[4, :9] = torch.tensor([6, 7.5, -5, 0.25, 0.75, 1.25, 1.75, 2.5, -0.1])
    x[5, 1] = -0.0
    x[6, 0] = 2.0 ** -126
    x[7, 0] = 2.0 ** -149
    code, byte = mx.encode(_np(x))
    for transpose in (False, True):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        codes, scales = megamoe.quantize_mxfp4(x.cuda(), transpose=transpose, status=status)
        ref = (code, byte) if not transpose else mx.encode(np.pad(_np(x).T, ((0, 0), (0, 24))))
        assert np.array_equal(codes.cpu().numpy(), mx.pack(ref[0]))
        assert np.array_equal(scales.cpu().numpy(), ref[1])
        assert status.item() == megamoe.DEV_NONFINITE
        v = _np(megamoe.dequantize_mxfp4(codes, scales, dtype=torch.float32))
        assert np.array_equal(v, mx.decode(*ref), equal_nan=True)
    assert byte[2].tolist() == [255, 125] and byte[3].tolist() == [0, 255]


def test_empty(cuda_lib):
    codes, scales = megamoe.quantize_mxfp4(torch.empty(0, 64, device="cuda"))
    assert codes.shape == (0, 32) and scales.shape == (0, 2)
    assert megamoe.dequantize_mxfp4(codes, scales).shape == (0, 64)
    w = megamoe.MxLinearWeights.quantize(torch.ones(32, 64, device="cuda"))
    out, _ = megamoe.linear_mxfp4(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), w)
    assert out.shape == (0, 32)
    gx, gw, _ = megamoe.linear_mxfp4_backward(torch.empty(0, 32, device="cuda"),
                                              torch.empty(0, 64, device="cuda"),
                                              torch.ones(32, 64, device="cuda"))
    assert gx.shape == (0, 64) and not gw.any() and gw.shape == (32, 64)


@pytest.mark.parametrize("T", [1, 2, 31, 33, 64, 65, 129, 300])
@pytest.mark.parametrize("K,N", [(32, 32), (96, 160), (256, 128), (1536, 2048), (7168, 96),
                                 (480, 800)])
def test_linear(cuda_lib, T, K, N):
    x = _x(T, K, seed=T)
    w = _x(N, K, seed=N + 1, wide=False)
    wq = mx.round_to_mx(_np(w))
    code, byte = mx.encode(_np(w))
    weights = megamoe.MxLinearWeights.prepare(torch.from_numpy(mx.pack(code)).cuda(),
                                              torch.from_numpy(byte).cuda())
    for epi, dt in ((megamoe.EPI_F32, torch.float32), (megamoe.EPI_BF16, torch.bfloat16)):
        out, ws = megamoe.linear_mxfp4(x.cuda(), weights, out_dtype=epi)
        assert out.dtype == dt
        _check_product(out, mx.round_to_mx(_np(x)), wq, dt)
        assert ws[:4].view(torch.int32).item() == 0
        # the workspace again, a strided output
        wide = torch.full((T, N + 8), 5.0, dtype=dt, device="cuda")
        again, _ = megamoe.linear_mxfp4(x.cuda(), weights, out_dtype=epi, out=wide[:, :N], ws=ws)
        assert torch.equal(again, out) and (wide[:, N:] == 5).all()


@pytest.mark.parametrize("T,K,N", [(4096, 512, 4096), (2050, 1024, 8224), (700, 7168, 2048)])
def test_linear_large_tiles(cuda_lib, T, K, N):
    """Sizes whose tiles fill the GPU, against fp32 products of the values on
    the GPU (TF32 off: both sides are fp32 sums of the same exact terms, so the
    bound holds twice)."""
    x, w = _x(T, K, seed=1).cuda(), _x(N, K, seed=2, wide=False).cuda()
    weights = megamoe.MxLinearWeights.quantize(w)
    out, _ = megamoe.linear_mxfp4(x, weights, out_dtype=megamoe.EPI_F32)
    xq = megamoe.dequantize_mxfp4(*megamoe.quantize_mxfp4(x), dtype=torch.float32)
    wq = megamoe.dequantize_mxfp4(*megamoe.quantize_mxfp4(w), dtype=torch.float32)
    want = xq @ wq.t()
    bound = 2 * (K / 64 + 18) * U * (xq.abs() @ wq.abs().t())
    assert ((out - want).abs() <= bound).all()


@pytest.mark.parametrize("T,K,N", [(4400, 320, 1312), (4700, 2080, 1536)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_bands_of_large_tiles(cuda_lib, T, K, N, dtype):
    """More than 16 rows of 256-row tiles, the last band of them and the last row
    of a tile not full, a ragged last K step; the bounds of the test above, with
    the output's own rounding."""
    x, w = _x(T, K, seed=1).cuda(), _x(N, K, seed=2, wide=False).cuda()
    weights = megamoe.MxLinearWeights.quantize(w)
    epi = megamoe.EPI_F32 if dtype == torch.float32 else megamoe.EPI_BF16
    wide = torch.full((T + 1, N + 8), 5.0, dtype=dtype, device="cuda")
    out, _ = megamoe.linear_mxfp4(x, weights, out_dtype=epi, out=wide[:T, :N])
    xq = megamoe.dequantize_mxfp4(*megamoe.quantize_mxfp4(x), dtype=torch.float32)
    wq = megamoe.dequantize_mxfp4(*megamoe.quantize_mxfp4(w), dtype=torch.float32)
    want = xq @ wq.t()
    bound = 2 * (K / 64 + 18) * U * (xq.abs() @ wq.abs().t())
    if dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (want.abs() + bound)
    assert ((out.float() - want).abs() <= bound).all()
    assert (wide[T] == 5).all() and (wide[:, N:] == 5).all()


def test_large_gradients(cuda_lib):
    """Both gradients on pairs of CTAs, a number of tokens that fills no K step."""
    T, K, N = 2600, 4160, 2080
    x, w, g = _x(T, K, seed=3).cuda(), _x(N, K, seed=4, wide=False).cuda(), _x(T, N, seed=5).cuda()

    def values(v, transpose=False):
        return megamoe.dequantize_mxfp4(*megamoe.quantize_mxfp4(v, transpose=transpose),
                                        dtype=torch.float32)

    for gx_dt, gw_dt in ((torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)):
        gx, gw, ws = megamoe.linear_mxfp4_backward(g, x, w, gx_dt, gw_dt)
        assert ws[:4].view(torch.int32).item() == 0
        for got, a, b in ((gx, values(g), values(w, True)), (gw, values(g, True), values(x, True))):
            want = a @ b.t()
            bound = 2 * (a.shape[1] / 64 + 18) * U * (a.abs() @ b.abs().t())
            if got.dtype == torch.bfloat16:
                bound = bound + 2.0 ** -8 * (want.abs() + bound)
            assert ((got.float() - want).abs() <= bound).all()


@pytest.mark.parametrize("T,K,N", [(1, 32, 32), (33, 96, 160), (64, 1536, 256), (333, 512, 800),
                                   (31, 2048, 96), (1000, 288, 480)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_gradients(cuda_lib, T, K, N, dtype):
    x, w, g = _x(T, K, dtype, 3), _x(N, K, dtype, 4, wide=False), _x(T, N, dtype, 5)
    rows, cols = mx.round_to_mx, mx.round_columns
    for gx_dt, gw_dt in ((torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)):
        gx, gw, ws = megamoe.linear_mxfp4_backward(g.cuda(), x.cuda(), w.cuda(), gx_dt, gw_dt)
        _check_product(gx, rows(_np(g)), cols(_np(w)), gx_dt)
        _check_product(gw, cols(_np(g)), cols(_np(x)), gw_dt)
        assert ws[:4].view(torch.int32).item() == 0
    only, none, _ = megamoe.linear_mxfp4_backward(g.cuda(), x.cuda(), w.cuda(), gx_dt, need_w=False)
    assert none is None and torch.equal(only, gx)
    none, only, _ = megamoe.linear_mxfp4_backward(g.cuda(), x.cuda(), w.cuda(), grad_w_dtype=gw_dt,
                                                  need_x=False)
    assert none is None and torch.equal(only, gw)


def test_linear_gradients_are_differences_where_rounding_is_exact(cuda_lib):
    """On E2M1 values with a 4 or 6 in each block the rounding is the identity,
    and unit steps of the loss sum(g * (x w^T)) are its derivatives exactly."""
    rng = np.random.default_rng(6)
    T, K, N = 64, 96, 32

    def grid(r, c):
        v = rng.choice(mx.GRID, (r, c)) * rng.choice([-1, 1], (r, c))
        v[::7, :] = 4.0
        v[:, ::7] = 6.0
        return v

    x, w, g = grid(T, K), grid(N, K), grid(T, N)
    t = lambda v: torch.tensor(v, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    gx, gw, _ = megamoe.linear_mxfp4_backward(t(g), t(x), t(w), torch.float32, torch.float32)
    loss = lambda a, b: (g * (a @ b.T)).sum()  # noqa: E731
    for r, c in ((0, 0), (3, 5), (31, 95), (17, 40)):
        step = np.zeros((T, K))
        step[r, c] = 1
        assert loss(x + step, w) - loss(x, w) == gx[r, c].item()
        assert loss(x, w + step[:N]) - loss(x, w) == gw[r, c].item()


# one launch; a tile a cluster, flipped and not; pairs of CTAs
@pytest.mark.parametrize("T,K,N", [(3, 64, 32), (50, 2048, 96), (100, 64, 160), (4096, 64, 2560)])
def test_non_finite_inputs_reach_the_output(cuda_lib, T, K, N):
    x = _x(T, K)
    x[1, 3] = torch.inf
    w = _x(N, K, seed=1, wide=False).cuda()
    out, ws = megamoe.linear_mxfp4(x.cuda(), megamoe.MxLinearWeights.quantize(w))
    good = torch.ones(T, dtype=torch.bool)
    good[1] = False
    assert torch.isnan(out[1]).all() and torch.isfinite(out[good.cuda()]).all()
    assert ws[:4].view(torch.int32).item() == megamoe.DEV_NONFINITE
    g = _x(T, N, seed=2).cuda()
    gx, gw, ws = megamoe.linear_mxfp4_backward(g, x.cuda(), w)
    assert torch.isfinite(gx).all() and torch.isnan(gw[:, 3]).all()
    assert torch.isfinite(gw[:, 4:]).all()
    assert ws[:4].view(torch.int32).item() == megamoe.DEV_NONFINITE
    # the next call clears the word
    x[1, 3] = 0
    _, _, ws = megamoe.linear_mxfp4_backward(g, x.cuda(), w, ws=ws)
    assert ws[:4].view(torch.int32).item() == 0


@pytest.mark.parametrize("T,K,N", [(3, 2048, 96), (50, 2048, 96), (100, 512, 160), (4096, 512, 2560)])
def test_waits_that_run_out_are_reported(cuda_lib, T, K, N):
    """A limit that no load meets: the kernels give up, report it and return,
    and the next call is right."""
    x, w = _x(T, K).cuda(), _x(N, K, seed=1, wide=False).cuda()
    weights = megamoe.MxLinearWeights.quantize(w)
    want, _ = megamoe.linear_mxfp4(x, weights)
    torch.cuda.synchronize()
    megamoe.set_wait_limit_ns(100)
    try:
        _, ws = megamoe.linear_mxfp4(x, weights)
        torch.cuda.synchronize()
        assert ws[:4].view(torch.int32).item() == megamoe.DEV_TIMEOUT
    finally:
        megamoe.set_wait_limit_ns(0)
    out, ws = megamoe.linear_mxfp4(x, weights, ws=ws)
    assert ws[:4].view(torch.int32).item() == 0 and torch.equal(out, want)


def _experts(E, d, I, seed):
    rng = np.random.default_rng(seed)
    raw, values = {}, {}
    for name, shape in (("w13", (E, 2 * I, d)), ("w2", (E, d, I))):
        code, byte = mx.encode(rng.standard_normal(shape).astype(np.float32) * 0.02)
        raw[name + "_codes"] = torch.from_numpy(mx.pack(code)).cuda()
        raw[name + "_scales"] = torch.from_numpy(byte).cuda()
        values[name] = mx.decode(code, byte)
    return megamoe.MxWeights.prepare(raw), values


# the intermediate's rounding to MXFP4 is decided on fp32 sums, so a value on
# the edge of two codes may fall either way; it is one term of I in an output:
# the framework's bound for a forward (helpers.py) holds
@pytest.mark.parametrize("T,E,k,d,I,pad", [(1, 8, 2, 256, 256, 32), (64, 8, 2, 256, 512, 32),
                                           (5, 33, 8, 512, 256, 128), (300, 8, 3, 256, 256, 32),
                                           (700, 8, 2, 512, 768, 64), (130, 3, 1, 256, 256, 32),
                                           (331, 8, 3, 256, 512, 96)])
def test_experts(cuda_lib, T, E, k, d, I, pad):
    weights, values = _experts(E, d, I, T)
    rng = np.random.default_rng(T + E)
    x = torch.tensor(rng.standard_normal((T, d)) * 0.5, dtype=torch.bfloat16)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[rng.random((T, k)) < 0.1] = -1
    if T > 2:
        ids[1] = -1  # a token without an expert
    w = rng.random((T, k)).astype(np.float32)
    fwd = megamoe.MxForward(weights, T, k, pad)
    for _ in range(2):
        out = fwd(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda())
        assert fwd.read_status() == 0
    want = mx.forward(_np(x), ids, w.astype(np.float64), values["w13"], values["w2"])
    assert_close_bf16(_np(out), want, what="mxfp4 experts")
    if T > 2:
        assert not out[1].any()


@pytest.mark.parametrize("T,E,k", [(1024, 48, 4), (1023, 48, 4), (700, 64, 6), (2100, 8, 2),
                                   (300, 16, 16)])
def test_experts_routed_over_many_blocks(cuda_lib, T, E, k):
    """Around and past the number of slots from which the routing takes several
    blocks, on single CTAs and on pairs; one expert without rows; 16 slots."""
    weights, values = _experts(E, 256, 256, E)
    rng = np.random.default_rng(T)
    x = torch.tensor(rng.standard_normal((T, 256)) * 0.5, dtype=torch.bfloat16)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[ids == 3] = -1
    w = rng.random((T, k)).astype(np.float32)
    fwd = megamoe.MxForward(weights, T, k)
    out = fwd(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda())
    assert fwd.read_status() == 0
    want = mx.forward(_np(x), ids, w.astype(np.float64), values["w13"], values["w2"])
    assert_close_bf16(_np(out), want, what="mxfp4 experts")
    assert torch.equal(out, fwd(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()))


@pytest.mark.parametrize("T,dtype", [(1, torch.float32), (40, torch.bfloat16), (600, torch.float32)])
def test_layer_from_logits_is_router_then_experts(cuda_lib, T, dtype):
    E, k, d, I = 16, 4, 256, 256
    weights, _ = _experts(E, d, I, 7)
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, d, generator=g).to(torch.bfloat16).cuda()
    logits = torch.randn(T, E, generator=g).to(dtype).cuda()
    logits[:, 3] = -torch.inf
    logits[0, 2:] = -torch.inf  # fewer experts than slots
    bias = (torch.arange(E) / 1024).cuda()
    how = dict(score="sigmoid", bias=bias, n_group=4, topk_group=2, scale=2.5)
    fwd = megamoe.MxForward(weights, T, k)
    ids, w = megamoe.router_scored_topk(logits, k, **how)
    want = fwd(x, ids, w).clone()
    got = fwd.from_logits(x, logits, **how)
    assert fwd.read_status() == 0 and torch.equal(got, want)
    assert torch.isfinite(got).all() and got.any()


def test_experts_bad_id_is_flagged_and_graph_replay_matches(cuda_lib):
    weights, _ = _experts(8, 256, 256, 9)
    x = _x(4, 256, seed=1).cuda()
    ids = torch.tensor([[0, 1], [2, 3], [4, 5], [6, 7]], dtype=torch.int32, device="cuda")
    w = torch.rand(4, 2, device="cuda")
    fwd = megamoe.MxForward(weights, 4, 2)
    want = fwd(x, ids, w).clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fwd(x, ids, w)
    fwd.out.zero_()
    g.replay()
    assert torch.equal(fwd.out[:4], want)
    bad = ids.clone()
    bad[1, 1] = 8
    fwd(x, bad, w)
    assert fwd.read_status() == megamoe.DEV_BAD_EXPERT_ID


@pytest.mark.parametrize("T", [6, 300, 400])
def test_non_finite_experts_reach_their_tokens_alone(cuda_lib, T):
    """Inf in one token and NaN scales in one expert's down rows: only the
    outputs that use them are not finite (small and large batches)."""
    E, k, d, I = 8, 3, 256, 256
    weights, values = _experts(E, d, I, 11)
    rng = np.random.default_rng(T)
    x = torch.tensor(rng.standard_normal((T, d)), dtype=torch.bfloat16)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    w = rng.random((T, k)).astype(np.float32) + 0.1
    fwd = megamoe.MxForward(weights, T, k)
    want = fwd(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()).clone()
    x[2, 7] = torch.inf
    got = fwd(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda())
    assert fwd.read_status() == megamoe.DEV_NONFINITE
    keep = torch.ones(T, dtype=torch.bool)
    keep[2] = False
    assert torch.isnan(got[2]).all() and torch.isfinite(got[keep.cuda()]).all()
    # a group of 16 rows that holds the token is stored as fp16: its other rows
    # carry that rounding
    assert_close_bf16(_np(got)[keep.numpy()], _np(want)[keep.numpy()], what="other tokens")
