"""The scored router where 32-bit scores are far apart in exponent or close in
value, against the order of the logits and 64-bit formulas; no token is drawn
again.

Two fp32 logits that differ at all differ by at least 2^-24 |l|, so for |l| >= 20
their scores, exp(l) times a common factor, differ by 16 units of 2^-23 and more,
several times what an fp32 exponential and division are off by: the choice is by
the logits, and only equal logits tie.  That holds for scores below the smallest
normal number too, as long as they have a few bits.

A weight is within (24 + span) 2^-23 of its value, relatively, span being the
largest distance of the logits from the one that exponentials are taken from; a
gradient's factors likewise, so each element is within (64 + 2 span) 2^-23 of
scale max|g| times its own p (1 - s) or s (1 - s)."""

import numpy as np
import pytest
import torch

from oracle import scored_router as sr
from nvfp4_block_scaled_topk_gb300 import megamoe

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


def _by_logit(l, k):
    return np.argsort(-l.astype(np.float64), axis=1, kind="stable")[:, :k]


def _neighbours(base, T, E, seed):
    """Logits within 200 units in the last place above base."""
    rng = np.random.default_rng(seed)
    step = np.spacing(np.float32(abs(base)))
    return (np.float32(base) + step * rng.integers(0, 200, (T, E))).astype(np.float32)


@pytest.mark.parametrize("base", [-24.0, -40.0, -72.0, -84.0])
@pytest.mark.parametrize("E", [64, 100, 384])
def test_neighbouring_logits_sigmoid(cuda_lib, base, E):
    l = _neighbours(base, 300, E, E)
    for dtype in (torch.float32,):
        ids, _ = megamoe.router_scored_topk(torch.from_numpy(l).to(dtype).cuda(), 8)
        assert np.array_equal(ids.cpu().numpy(), _by_logit(l, 8))


@pytest.mark.parametrize("base", [-24.0, -40.0, -72.0, -84.0])
@pytest.mark.parametrize("E", [64, 100, 384])
def test_neighbouring_logits_softmax(cuda_lib, base, E):
    l = _neighbours(base, 300, E, E + 1)
    l[:, 5] = 0
    ids, _ = megamoe.router_scored_topk(torch.from_numpy(l).cuda(), 8, "softmax")
    assert np.array_equal(ids.cpu().numpy(), _by_logit(l, 8))


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
def test_scores_below_the_smallest_normal_number(cuda_lib, kind):
    l = np.linspace(-98, -89, 19, dtype=np.float32)[None]  # the lower index scores less
    if kind == "softmax":
        l = np.concatenate([np.zeros((1, 1), np.float32), l], 1)
    ids, _ = megamoe.router_scored_topk(torch.from_numpy(l).cuda(), 12, kind)
    assert np.array_equal(ids.cpu().numpy(), _by_logit(l, 12))


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("group_top", [1, 2])
def test_groups_ranked_by_small_scores(cuda_lib, kind, group_top):
    """Five groups of four; all but the first lie within units of each other, then
    below the smallest normal number."""
    for base, step in ((-72.0, np.spacing(np.float32(72.0))), (-97.0, 0.5)):
        l = np.full((1, 20), -150.0, np.float32)
        l[0, 1] = 0
        for group, place in ((1, 3), (2, 0), (3, 2), (4, 1)):
            l[0, 4 * group + 2] = np.float32(base + place * step)
        ids, _ = megamoe.router_scored_topk(torch.from_numpy(l).cuda(), 3, kind, n_group=5,
                                            topk_group=3, group_top=group_top)
        assert ids.tolist() == [[1, 6, 14]]


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
def test_many_tied_neighbours(cuda_lib, kind):
    """More equal scores than lanes, next to larger and smaller ones by one unit."""
    step = np.spacing(np.float32(48.0))
    l = np.full((2, 200), np.float32(-48.0), np.float32)
    l[0, 150], l[0, 60] = -48 + 2 * step, -48 + step
    l[1, :100] = -48 - step
    if kind == "softmax":
        l[:, 199] = 0
    ids, _ = megamoe.router_scored_topk(torch.from_numpy(l).cuda(), 6, kind)
    assert np.array_equal(ids.cpu().numpy(), _by_logit(l, 6))


def test_weights_of_small_scores(cuda_lib):
    """Without renormalisation the weights are the scores, subnormal ones to their
    last bit or two."""
    l = np.linspace(-98, -60, 16, dtype=np.float32)[None]
    ids, w = megamoe.router_scored_topk(torch.from_numpy(l).cuda(), 16, renormalize=False)
    want = sr.weigh(l[0], ids[0].tolist(), "sigmoid", renormalize=False)
    tol = (24 + 98) * U * want + 2 * 2.0 ** -149
    assert (np.abs(w[0].double().cpu().numpy() - want) <= tol).all()


def test_scores_keep_the_order_of_the_logits(cuda_lib):
    """All of 16 experts taken: where scores near one are few units apart, the larger
    logit's is not the smaller, and equal scores come by index."""
    rng = np.random.default_rng(4)
    l = rng.uniform(4, 18, (4000, 1)) + rng.uniform(0, 1, (4000, 16)) * np.exp2(
        rng.integers(-14, 1, (4000, 1)))
    l = l.astype(np.float32)
    ids, w = megamoe.router_scored_topk(torch.from_numpy(l).cuda(), 16, renormalize=False)
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    taken = np.take_along_axis(l, ids, 1)
    before = (taken[:, :-1] > taken[:, 1:]) | ((w[:, :-1] == w[:, 1:]) & (ids[:, :-1] < ids[:, 1:]))
    assert (w[:, :-1] >= w[:, 1:]).all() and before.all()
    want = 1 / (1 + np.exp(-taken.astype(np.float64)))
    assert (np.abs(w - want) <= 4 * U * want).all()


@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_of_confident_scores(cuda_lib, renormalize):
    """1 - s of logits of 10 to 40 is e^-l, not what is left of s after its rounding."""
    rng = np.random.default_rng(8)
    l = rng.uniform(10, 40, (50, 12)).astype(np.float32)
    l[1::2] *= -1
    l[::5, 3] *= -1
    ids, _ = megamoe.router_scored_topk(torch.from_numpy(l).cuda(), 6)
    g = rng.standard_normal((50, 6)).astype(np.float32)
    got = megamoe.router_scored_topk_backward(torch.from_numpy(l).cuda(), ids,
                                              torch.from_numpy(g).cuda(), renormalize=renormalize,
                                              scale=2.5)
    at = ids.cpu().numpy()
    x, g = np.take_along_axis(l, at, 1).astype(np.float64), g.astype(np.float64)
    e = np.exp(-np.abs(x))
    s, rest = np.where(x >= 0, 1, e) / (1 + e), np.where(x >= 0, e, 1) / (1 + e)
    if renormalize:
        p = s / s.sum(1, keepdims=True)
        factor, dl = p * rest, p * rest * (g - (g * p).sum(1, keepdims=True))
    else:
        factor, dl = s * rest, s * rest * g
    want, bound = np.zeros(l.shape), np.zeros(l.shape)
    np.put_along_axis(want, at, 2.5 * dl, 1)
    most = np.abs(g).max(1, keepdims=True)
    np.put_along_axis(bound, at, (64 + 2 * 40) * U * 2.5 * most * factor, 1)
    assert (np.abs(got.double().cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_renormalised_softmax_far_below_the_top(cuda_lib, dtype):
    """The bias takes experts whose softmax scores are nothing in fp32: their weights
    are shares of one another all the same, and the gradient is that of these."""
    rng = np.random.default_rng(9)
    T, E, k = 40, 24, 4
    l = torch.tensor(rng.uniform(-60, 60, (T, E)), dtype=dtype)
    l[:, :8] -= 130  # 70 and more below the others
    l[0, :8] = -float(np.finfo(np.float32).max) if dtype == torch.float32 else -3e38
    bias = np.where(np.arange(E) < 8, 4 + np.arange(E) / 8, 0)
    kw = dict(score="softmax", scale=2.5)
    ids, w = megamoe.router_scored_topk(l.cuda(), k, bias=torch.tensor(bias, dtype=torch.float32).cuda(),
                                        **kw)
    assert (ids.cpu().numpy() == [7, 6, 5, 4]).all()
    g = torch.tensor(rng.standard_normal((T, k)), dtype=torch.float32)
    got = megamoe.router_scored_topk_backward(l.cuda(), ids, g.cuda(), **kw)
    x, gd = l[:, [7, 6, 5, 4]].double().numpy(), g.double().numpy()
    p = np.exp(x - x.max(1, keepdims=True))
    p = p / p.sum(1, keepdims=True)
    assert (np.abs(w.double().cpu().numpy() - 2.5 * p) <= (24 + 120) * U * 2.5 * p + 1e-44).all()
    want = np.zeros((T, E))
    want[:, [7, 6, 5, 4]] = 2.5 * p * (gd - (gd * p).sum(1, keepdims=True))
    bound = (64 + 2 * 120) * U * 2.5 * np.abs(gd).max(1, keepdims=True) + np.abs(want) * (
        2.0 ** -8 if dtype == torch.bfloat16 else 0)
    assert (np.abs(got.double().cpu().numpy() - want) <= bound).all()
