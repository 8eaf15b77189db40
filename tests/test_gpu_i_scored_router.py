"""megamoe_router_scored_topk and its gradient against the float64 oracle:
sizes, groups, types, strides, masked and tied experts.

Ids have to be equal, so the inputs are drawn with a margin: a token whose
choice hangs on two scores closer than 2e-6 (relative) is drawn again; equal
logits under equal biases are real ties and stay.

Tolerances.  exp(l - m) carries the rounding of its argument, |l - m| 2^-24,
and 2 units of its own; the division, the sum of up to 16 weights and the
scale add at most 20 units of 2^-24: a weight is within
(24 + max |l - m|) 2^-23 of its value, relatively.  A gradient is a product of
such terms with sums over the k incoming gradients: within
(64 + 2 max |l - m|) 2^-23 scale max|g| of its value."""

import numpy as np
import pytest
import torch

from oracle import scored_router as sr
from nvfp4_block_scaled_topk_gb300 import megamoe

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


def _contested(l, k, kind, bias, n_group, topk_group, group_top):
    s, alive = sr.scores(l, kind)
    c = np.where(alive, s if bias is None else s + bias, -np.inf)

    def close(v):
        v = np.sort(v[np.isfinite(v)])[::-1]
        gap = v[:-1] - v[1:]
        return ((gap > 0) & (gap < 2e-6 * np.maximum(abs(v[:-1]), abs(v[1:])))).any()

    groups = c.reshape(n_group, -1)
    best = [sum(sorted(g[np.isfinite(g)])[::-1][:group_top]) for g in groups]
    return close(c) or close(np.array(best))


def _draw(T, E, kind, dtype, seed, bias=None, masked=0, k=1, spread=1.5, **groups):
    g = torch.Generator().manual_seed(seed)
    out = torch.zeros(T, E, dtype=dtype)
    for t in range(T):
        for _ in range(100):
            l = (torch.randn(E, generator=g) * spread).to(dtype)
            if masked:
                l[torch.randperm(E, generator=g)[:masked]] = -torch.inf
            if not _contested(l.double().numpy(), k, kind, bias, groups["n_group"],
                              groups["topk_group"], groups["group_top"]):
                break
        out[t] = l
    return out


def _span(l):
    v = l.double().numpy()
    v = v[np.isfinite(v)]
    return float(v.max() - v.min()) if v.size else 0.0


CASES = [
    # T, E, k, kind, bias, n_group, topk_group, group_top, renormalize, dtype, masked
    (1, 384, 6, "sigmoid", True, 8, 4, 2, True, torch.float32, 0),
    (33, 384, 6, "sigmoid", True, 8, 4, 2, True, torch.float32, 5),
    (5, 384, 8, "softmax", False, 1, 1, 2, False, torch.float32, 0),
    (17, 48, 6, "softmax", True, 4, 2, 1, True, torch.bfloat16, 3),
    (7, 1, 1, "sigmoid", False, 1, 1, 2, True, torch.float32, 0),
    (9, 33, 5, "softmax", False, 3, 2, 2, True, torch.float32, 0),
    (6, 1024, 16, "sigmoid", False, 1, 1, 2, True, torch.float32, 0),
    (4, 1020, 7, "sigmoid", True, 17, 5, 2, False, torch.float32, 100),
    (5, 64, 4, "sigmoid", False, 32, 3, 2, True, torch.bfloat16, 0),
    (8, 8, 8, "softmax", False, 1, 1, 2, True, torch.float32, 6),
    (3, 96, 8, "sigmoid", True, 8, 1, 2, True, torch.float32, 90),
]


@pytest.mark.parametrize("T,E,k,kind,bias,n_group,topk_group,group_top,renormalize,dtype,masked",
                         CASES)
def test_forward_and_gradient(cuda_lib, T, E, k, kind, bias, n_group, topk_group, group_top,
                              renormalize, dtype, masked):
    groups = dict(n_group=n_group, topk_group=topk_group, group_top=group_top)
    rng = np.random.default_rng(E + k)
    b = rng.integers(-24, 25, E) / 1024 if bias else None
    l = _draw(T, E, kind, dtype, seed=E * 3 + k, bias=b, masked=masked, k=k, **groups)
    want_ids, want_w = sr.router(l.double().numpy(), k, kind, b, renormalize=renormalize,
                                 scale=2.5, **groups)
    # rows of a wider matrix: a stride of its own
    wide = torch.full((T, E + 3), 99.0, dtype=dtype, device="cuda")
    wide[:, :E] = l.cuda()
    bt = None if b is None else torch.tensor(b, dtype=torch.float32, device="cuda")
    for logits in (l.cuda(), wide[:, :E]):
        ids, w = megamoe.router_scored_topk(logits, k, kind, bias=bt, renormalize=renormalize,
                                            scale=2.5, **groups)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        tol = (24 + _span(l)) * U
        assert np.allclose(w.cpu().numpy(), want_w, rtol=tol, atol=1e-37)
        grad = torch.tensor(rng.standard_normal((T, k)), dtype=torch.float32)
        got = megamoe.router_scored_topk_backward(logits, ids, grad.cuda(), kind,
                                                  renormalize=renormalize, scale=2.5)
        want = sr.backward(l.double().numpy(), want_ids, grad.double().numpy(), kind, renormalize,
                           2.5)
        assert got.dtype == dtype
        err = np.abs(got.double().cpu().numpy() - want)
        bound = (64 + 2 * _span(l)) * U * 2.5 * grad.abs().max().item()
        if dtype == torch.bfloat16:
            bound = bound + np.abs(want) * 2.0 ** -8
        assert (err <= bound).all(), err.max()


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
def test_ties_go_to_the_lower_index(cuda_lib, kind):
    l = torch.zeros(3, 40)
    l[1, 7::5] = 1.0
    l[2] = torch.arange(40).remainder(4).float()
    for n_group, topk_group in ((1, 1), (4, 2), (8, 3)):
        ids, _ = megamoe.router_scored_topk(l.cuda(), 6, kind, n_group=n_group,
                                            topk_group=topk_group)
        want, _ = sr.router(l.double().numpy(), 6, kind, n_group=n_group, topk_group=topk_group)
        assert np.array_equal(ids.cpu().numpy(), want)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_masked_rows_and_extreme_logits(cuda_lib, kind, renormalize):
    E = 16
    low = float(np.finfo(np.float32).min)
    l = torch.zeros(7, E)
    l[0] = -torch.inf                      # nothing to take
    l[1] = torch.nan                       # nothing to take
    l[2, 1:] = -torch.inf                  # one expert left
    l[3, 5], l[3, 6] = torch.inf, torch.nan
    l[4] = low                             # the type's lowest value: ordinary logits
    l[5, 3] = low
    l[6] = torch.linspace(-120, 120, E)
    ids, w = megamoe.router_scored_topk(l.cuda(), 4, kind, renormalize=renormalize)
    want_ids, want_w = sr.router(l.double().numpy(), 4, kind, renormalize=renormalize)
    if kind == "sigmoid":
        # scores within 2^-25 of one are one in 32 bits, ties: the first four
        # of the logits past 25 ln 2 = 17.4, which here are 24, 40, 56, ...
        want_ids[6], want_w[6] = [9, 10, 11, 12], want_w[6].mean()
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert np.allclose(w.cpu().numpy(), want_w, rtol=260 * U, atol=1e-37)
    g = torch.ones(7, 4) * torch.tensor([1.0, -2.0, 3.0, 0.5])
    got = megamoe.router_scored_topk_backward(l.cuda(), ids, g.cuda(), kind,
                                              renormalize=renormalize)
    want = sr.backward(l.double().numpy(), want_ids, g.double().numpy(), kind, renormalize)
    assert np.isfinite(got.cpu().numpy()).all()
    assert (np.abs(got.double().cpu().numpy() - want) <= (64 + 2 * 240) * U * 3).all()
    assert ids[0].tolist() == [-1] * 4 and w[0].tolist() == [0] * 4 and not got[:2].any()


def test_bias_excludes_and_moves_only_the_choice(cuda_lib):
    l = torch.tensor([[0.5, 0.25, 0.0, -0.5]]).cuda()
    bias = torch.tensor([-torch.inf, 0.0, torch.nan, 10.0]).cuda()
    ids, w = megamoe.router_scored_topk(l, 3, bias=bias, renormalize=False)
    assert ids.tolist() == [[3, 1, -1]]
    s = 1 / (1 + np.exp([0.5, -0.25]))
    assert np.allclose(w[0].tolist(), [*s, 0], rtol=24 * U)


def test_zero_tokens_and_another_stream(cuda_lib):
    ids, w = megamoe.router_scored_topk(torch.empty(0, 8, device="cuda"), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    g = megamoe.router_scored_topk_backward(torch.empty(0, 8, device="cuda"), ids, w)
    assert g.shape == (0, 8)
    l = torch.randn(2000, 384, device="cuda")
    want = megamoe.router_scored_topk(l, 6, n_group=8, topk_group=4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = megamoe.router_scored_topk(l, 6, n_group=8, topk_group=4)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
