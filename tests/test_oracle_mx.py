"""Pins of the oracle's MXFP4 codec and scored router: hand tables, closed
forms, differences."""

import numpy as np
import pytest

from oracle import mxfp4 as mx
from oracle import scored_router as sr


def test_codec_by_hand():
    x = np.zeros(32)
    x[:9] = [6, 7.5, -5, 0.25, 0.75, 1.25, 1.75, 2.5, -0.1]
    code, byte = mx.encode(x)
    assert byte.tolist() == [127]  # amax 7.5: floor(log2) - 2 = 0
    # 7.5 saturates; 5, 0.25, 0.75, ... are midpoints, to the even code
    assert code[:9].tolist() == [7, 7, 8 + 6, 0, 2, 2, 4, 4, 8]
    assert mx.decode(code, byte)[:9].tolist() == [6, 6, -4, 0, 1, 1, 2, 2, 0]


@pytest.mark.parametrize("e", [-130, -127, -126, -125, -1, 0, 20, 127])
def test_scale_of_a_power_of_two(e):
    x = np.zeros(32)
    x[3] = np.ldexp(1.0, e)
    code, byte = mx.encode(x)
    assert byte[0] == max(e - 2, -127) + 127
    if e >= -125:
        assert code[3] == 6 and mx.decode(code, byte)[3] == x[3]  # 4 * 2^(e - 2)


def test_zero_and_non_finite_blocks():
    x = np.zeros((3, 32))
    x[1, 4], x[2, 5] = np.inf, np.nan
    code, byte = mx.encode(x)
    assert byte.ravel().tolist() == [0, 255, 255] and not code.any()
    assert np.isnan(mx.decode(code, byte)[1:]).all()


def test_grid_values_survive_and_errors_are_bounded():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((64, 96)).astype(np.float32)
    v = mx.round_to_mx(x)
    assert np.array_equal(mx.round_to_mx(v), v)
    amax = np.abs(x).reshape(64, 3, 32).max(-1).repeat(32, -1)
    # half a step below 6 scales, a quarter of amax past them
    assert (np.abs(v - x) <= amax / 4).all()
    assert np.array_equal(mx.unpack(mx.pack(mx.encode(x)[0])), mx.encode(x)[0])


def test_atoms_by_index():
    rows, blocks = 200, 11
    s = np.arange(rows * blocks, dtype=np.int64).reshape(rows, blocks).astype(np.uint8)
    a = mx.atoms(s)
    assert a.size == 256 * 16
    for r, b in ((0, 0), (31, 3), (32, 4), (127, 10), (199, 10)):
        at = ((r // 128) * 4 + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4
        assert a[at] == s[r, b]


def test_router_by_hand():
    l = np.array([0.0, 2.0, 1.0, 2.0, -np.inf, 5.0, np.nan, -1.0])
    # groups {0,1} {2,3} {4,5} {6,7}: sums of the two best sigmoids 1.38, 1.61,
    # 0.99, 0.27; of the best one 0.88, 0.88, 0.99, 0.27 (the tie to group 0)
    assert sr.choose(l, 3, "sigmoid", n_group=4, topk_group=2) == [1, 3, 2]
    assert sr.choose(l, 3, "sigmoid", n_group=4, topk_group=2, group_top=1) == [5, 1, 0]
    assert sr.choose(l, 8, "softmax") == [5, 1, 3, 2, 0, 7, -1, -1]
    bias = np.zeros(8)
    bias[7] = 1.0
    assert sr.choose(l, 2, "sigmoid", bias=bias) == [7, 5]
    w = sr.weigh(l, [7, 5, -1], "sigmoid")
    s = 1 / (1 + np.exp([1.0, -5.0]))
    assert np.allclose(w, [*(s / s.sum()), 0])
    assert sr.choose(np.full(4, -np.inf), 2, "softmax") == [-1, -1]
    assert np.allclose(sr.weigh(l, [0, 1], "softmax", renormalize=False, scale=2).sum(),
                       2 * (1 + np.exp(2)) / (1 + 2 * np.exp(2) + np.exp(1) + np.exp(5) + np.exp(-1)))


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_router_gradient_is_the_difference_quotient(kind, renormalize):
    rng = np.random.default_rng(1)
    l = rng.standard_normal((3, 10)) * 2
    l[0, 4] = -np.inf
    ids, _ = sr.router(l, 4, kind)
    ids[1, 3] = -1
    g = rng.standard_normal((3, 4))
    got = sr.backward(l, ids, g, kind, renormalize, 2.5)

    def loss(v):
        return sum((g[t] * sr.weigh(v[t], ids[t], kind, renormalize, 2.5)).sum() for t in range(3))

    h = 1e-5
    for t in range(3):
        for e in range(10):
            if not np.isfinite(l[t, e]):
                assert got[t, e] == 0
                continue
            up, down = l.copy(), l.copy()
            up[t, e] += h
            down[t, e] -= h
            # the quotient's own error is h^2 times a third derivative below 10
            assert abs((loss(up) - loss(down)) / (2 * h) - got[t, e]) < 1e-8


def test_linear_gradients_are_differences_where_rounding_is_exact():
    """On grid values with a 4 in each block of either direction the rounding
    is the identity, and the gradients are those of the plain product."""
    rng = np.random.default_rng(2)
    T, K, N = 32, 64, 32

    def grid(r, c):
        v = rng.choice(mx.GRID, (r, c)) * rng.choice([-1, 1], (r, c))
        v[::7, :] = 4.0
        v[:, ::7] = 6.0
        return v

    x, w, g = grid(T, K), grid(N, K), grid(T, N)
    gx, gw = mx.linear_backward(g, x, w)
    # the loss sum(g * (x w^T)) is linear in each element: unit steps give its
    # derivative exactly
    loss = lambda a, b: (g * (a @ b.T)).sum()  # noqa: E731
    for r, c in ((0, 0), (3, 5), (31, 63), (17, 40)):
        step = np.zeros((T, K))
        step[r, c] = 1
        assert loss(x + step, w) - loss(x, w) == gx[r, c]
        assert loss(x, w + step) - loss(x, w) == gw[r, c]
