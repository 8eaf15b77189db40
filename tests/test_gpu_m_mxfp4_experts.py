"""MXFP4 experts on tokens of very different sizes and beside tokens and weights
that are not finite, element by element against the float64 oracle.

Tolerance.  Only tokens are drawn whose intermediate h is rounded to MXFP4 the same
way whatever the error of the sums behind it: no |h| lies within its error of the
edge of two codes, no block's largest within its error of a power of two.  That
error comes from the fp32 sums of gate and up, (d / 64 + 18) 2^-23 sum |p q| each,
and SiLU's exponential and division, 2^-20 and (2 + |g|) 2^-21 of the share that the
exponential has.  Then the output is off by the down product's fp32 sum,
(I / 64 + 18) 2^-23 sum |p q|; by its 16-bit storage, half a unit of 2^-14 of the
largest of 32 neighbouring columns of the same row; and by its one rounding to
bf16.  Nothing in that depends on another token."""

import numpy as np
import pytest
import torch

from oracle import mxfp4 as mx
from nvfp4_block_scaled_topk_gb300 import megamoe
from helpers import bf16_half_ulp

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
E, D, I = 4, 256, 256
EDGES = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
# tokens, so that an expert has rows for: tiles of 32, of 64, token-major tiles, pairs
TOKENS = [24, 160, 360, 520]


def _np(t):
    return t.double().cpu().numpy()


def _weights(seed):
    rng = np.random.default_rng(seed)
    raw, values = {}, {}
    for name, shape in (("w13", (E, 2 * I, D)), ("w2", (E, D, I))):
        code, byte = mx.encode(rng.standard_normal(shape).astype(np.float32) * 0.02)
        raw[name + "_codes"] = torch.from_numpy(mx.pack(code)).cuda()
        raw[name + "_scales"] = torch.from_numpy(byte).cuda()
        values[name] = mx.decode(code, byte)
    return raw, values


def _intermediate(x, w13):
    """(h, its possible error) of tokens x [n, D] through one expert's w13."""
    xq = mx.round_to_mx(x)
    sums, off = xq @ w13.T, (D / 64 + 18) * U * (np.abs(xq) @ np.abs(w13).T)
    g, u, dg, du = sums[:, :I], sums[:, I:], off[:, :I], off[:, I:]
    with np.errstate(over="ignore"):
        share = 1 / (1 + np.exp(g))  # of the exponential in 1 + exp(-g)
        s = g / (1 + np.exp(-g))
    ds = 1.1 * dg + np.abs(s) * (2.0 ** -20 + (2 + np.abs(g)) * 2.0 ** -21 * share) + 1e-35
    return s * u, np.abs(u) * ds + (np.abs(s) + ds) * du


def _settled(h, err):
    """Tokens whose every h is rounded the same way within its error."""
    b, e = np.abs(h).reshape(len(h), -1, 32), err.reshape(len(h), -1, 32)
    most = b.max(-1, keepdims=True)
    power = np.exp2(np.floor(np.log2(most)))
    scale = power / 4
    at_edge = (np.abs(b[..., None] / scale[..., None] - EDGES) <= (e / scale)[..., None]).any(-1)
    at_power = (most - power <= e) | (2 * power - most <= e)
    return ~(at_edge | at_power).any((1, 2))


def _tokens(T, values, sizes, seed):
    """T settled tokens and their experts; token t is of size sizes[t % len]."""
    rng = np.random.default_rng(seed)
    x, ids = np.zeros((T, D)), rng.integers(0, E, (T, 1)).astype(np.int32)
    left = np.arange(T)
    while len(left):
        t = torch.tensor(rng.standard_normal((len(left), D)) * np.resize(sizes, T)[left, None],
                         dtype=torch.bfloat16)
        x[left] = _np(t)
        fine = np.zeros(len(left), bool)
        for e in range(E):
            mine = ids[left, 0] == e
            if mine.any():
                fine[mine] = _settled(*_intermediate(x[left[mine]], values["w13"][e]))
        left = left[~fine]
    return x, ids, rng.random((T, 1)).astype(np.float32) + 0.5


def _expected(x, ids, w, values):
    """(output before its rounding, bound of the error without it, |y| of 32
    columns, by token)."""
    want, bound, group = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)
    for e in range(E):
        mine = ids[:, 0] == e
        if not mine.any():
            continue
        hq = mx.round_to_mx(_intermediate(x[mine], values["w13"][e])[0])
        y = hq @ values["w2"][e].T
        most = np.abs(y).reshape(len(y), -1, 32).max(-1).repeat(32, 1)
        wt = w[mine].astype(np.float64)
        want[mine] = wt * y
        bound[mine] = wt * ((I / 64 + 20) * U * (np.abs(hq) @ np.abs(values["w2"][e]).T)
                            + 2.0 ** -15 * 1.01 * most)
        group[mine] = wt * most
    return want, bound, group


def _check(got, want, bound, what=""):
    bound = bound + bf16_half_ulp(np.abs(want) + bound)
    err = np.abs(got - want)
    assert (err <= bound).all(), (what, (err / bound).max())


def _run(raw, x, ids, w):
    fwd = megamoe.MxForward(megamoe.MxWeights.prepare(raw), len(x), 1)
    out = fwd(torch.tensor(x, dtype=torch.bfloat16).cuda(), torch.from_numpy(ids).cuda(),
              torch.from_numpy(w).cuda())
    return _np(out), fwd.read_status()


@pytest.mark.parametrize("T", TOKENS)
def test_small_tokens_beside_large_ones(cuda_lib, T):
    raw, values = _weights(1)
    x, ids, w = _tokens(T, values, 2.0 ** -np.arange(11), T)
    got, status = _run(raw, x, ids, w)
    assert status == 0
    want, bound, _ = _expected(x, ids, w, values)
    _check(got, want, bound)


@pytest.mark.parametrize("T", TOKENS)
def test_large_tokens_beside_one_that_is_not_finite(cuda_lib, T):
    """Outputs past the largest 16-bit float, a NaN in another token of the same
    expert and 16 rows."""
    raw, values = _weights(2)
    x, ids, w = _tokens(T, values, [2.0 ** 11], T + 1)
    want, bound, _ = _expected(x, ids, w, values)
    assert np.abs(want).max() > 65536
    bad = np.flatnonzero(ids[:, 0] == 2)[0]
    x[bad, 7] = np.nan
    got, status = _run(raw, x, ids, w)
    assert status == megamoe.DEV_NONFINITE
    others = np.arange(T) != bad
    assert np.isnan(got[bad]).all()
    _check(got[others], want[others], bound[others])


@pytest.mark.parametrize("T", TOKENS)
def test_weights_that_are_not_finite(cuda_lib, T):
    """NaN scales in rows of one expert's down projection: NaN in those columns of
    the tokens of that expert alone; a rounding of bf16 more is allowed to the 31
    columns beside one in a row."""
    raw, values = _weights(3)
    x, ids, w = _tokens(T, values, [0.5, 8.0], T + 2)
    want, bound, group = _expected(x, ids, w, values)
    columns = [3, 100, 133]
    for i, c in enumerate(columns):
        raw["w2_scales"][1, c, i] = 255
    got, _ = _run(raw, x, ids, w)
    nan = np.zeros((T, D), bool)
    nan[np.ix_(ids[:, 0] == 1, columns)] = True
    assert np.array_equal(np.isnan(got), nan)
    beside = np.zeros((T, D // 32), bool)
    beside[np.ix_(ids[:, 0] == 1, np.array(columns) // 32)] = True
    bound = bound + np.where(beside.repeat(32, 1), 2.0 ** -9 * np.abs(want), 0)
    _check(got[~nan], want[~nan], bound[~nan])
