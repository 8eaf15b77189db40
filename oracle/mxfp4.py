"""MXFP4 of the oracle (test infrastructure only): E2M1 elements with one
power-of-two scale per 32, by the OCP Microscaling Formats specification 1.0
(section 6.3: the shared exponent is floor(log2(amax)) minus the largest
exponent of E2M1, 2; elements are rounded to nearest, ties to even, and
saturate).  Every step but the rounding is exact, so float64 reaches the same
bytes as any correct implementation.  Two readings the specification leaves
open: the scale is at least 2^-127 (byte 0), and a block holding Inf or NaN
gets the NaN scale (byte 255) and zero codes.
"""

from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 32
NAN_SCALE = 255


def encode(x):
    """x [..., K] (K a multiple of 32) -> (codes [..., K] 0..15, scale bytes
    [..., K / 32])."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    finite = np.isfinite(b).all(-1)
    amax = np.where(finite, np.abs(np.where(np.isfinite(b), b, 0)).max(-1), 0.0)
    _, e = np.frexp(amax)  # amax = m 2^e, m in [1/2, 1)
    exp = np.where(amax > 0, np.maximum(e - 1 - 2, -127), -127)
    r = np.abs(np.where(finite[..., None], b, 0)) * np.ldexp(1.0, -exp)[..., None]
    code = np.zeros(r.shape, np.uint8)
    for i in range(7):
        mid = (GRID[i] + GRID[i + 1]) / 2
        # past the midpoint, or on it with the lower code odd: the upper one
        code = np.where((r > mid) | ((r == mid) & (i % 2 == 1)), i + 1, code).astype(np.uint8)
    sign = np.where(finite[..., None], np.signbit(b), False)
    code |= sign.astype(np.uint8) << 3
    byte = np.where(finite, exp + 127, NAN_SCALE).astype(np.uint8)
    return code.reshape(x.shape), byte


def decode(codes, scales):
    """Values of codes [..., K] and scale bytes [..., K / 32]."""
    codes = np.asarray(codes)
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.ldexp(1.0, np.asarray(scales).astype(np.int64) - 127)
    s = np.where(np.asarray(scales) == NAN_SCALE, np.nan, s)
    return v * np.repeat(s, BLOCK, -1)


def round_to_mx(x):
    """x [..., K] as its MXFP4 values."""
    return decode(*encode(x))


def round_columns(x):
    """x [rows, K] -> values of x^T [K, R], quantised along the rows, R = rows
    up to a multiple of 32 (zeros past the last)."""
    t = np.asarray(x, dtype=np.float64).T
    return round_to_mx(np.pad(t, ((0, 0), (0, -t.shape[1] % BLOCK))))


def pack(codes):
    """Two codes per byte, the even element in the low nibble."""
    return (codes[..., ::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    return np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)


def atoms(scales):
    """Row-major scale bytes [rows, K / 32] -> the atom layout: atoms of 128
    rows x 4 blocks, byte 16 i + 4 j + b of atom (a, c) is row 128 a + 32 j + i,
    block 4 c + b; blocks padded to a multiple of 8, rows to 128, with zeros."""
    rows, blocks = scales.shape
    full = np.zeros((-(-rows // 128) * 128, -(-blocks // 8) * 8), np.uint8)
    full[:rows, :blocks] = scales
    a = full.reshape(full.shape[0] // 128, 4, 32, full.shape[1] // 4, 4)  # a, j, i, c, b
    return a.transpose(0, 3, 2, 1, 4).reshape(-1)


def linear(x, w_values):
    return round_to_mx(x) @ np.asarray(w_values, np.float64).T


def linear_backward(grad, x, w):
    """(grad_x, grad_w): each product's operands rounded along the dimension it
    sums over."""
    return (round_to_mx(grad) @ round_columns(w).T, round_columns(grad) @ round_columns(x).T)


def forward(x, ids, weights, w13, w2):
    """The routed experts: w13 [E, 2I, d] and w2 [E, d, I] values.  Returns
    (out [T, d], h of every slot before its rounding, for the tests)."""
    x = np.asarray(x, np.float64)
    T, k = ids.shape
    I = w2.shape[2]
    xq = round_to_mx(x)
    out = np.zeros_like(x)
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if e < 0:
                continue
            h = w13[e] @ xq[t]
            g, u = h[:I], h[I:]
            h = g / (1 + np.exp(-g)) * u
            out[t] += weights[t, j] * (w2[e] @ round_to_mx(h))
    return out
