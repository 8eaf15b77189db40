"""Scored router of the oracle (test infrastructure only), one token at a time
in float64: scores of every expert (sigmoid or softmax), the choice by score +
bias within the best groups, ties to the lower index, weights from the scores.
An expert whose logit is NaN or -inf, or whose score + bias is, is never taken;
+inf counts as the largest float32; slots left over get id -1, weight 0.
"""

from __future__ import annotations

import numpy as np

F32_MAX = float(np.finfo(np.float32).max)


def scores(l, kind):
    """Scores of one token's logits l [E]."""
    l = np.asarray(l, np.float64)
    alive = l > -np.inf
    v = np.where(alive, np.minimum(l, F32_MAX), 0.0)
    with np.errstate(over="ignore"):
        if kind == "sigmoid":
            s = 1 / (1 + np.exp(-v))
        else:
            ex = np.exp(v - v[alive].max()) if alive.any() else np.zeros_like(v)
            ex = np.where(alive, ex, 0.0)
            s = ex / ex.sum() if alive.any() else ex
    return np.where(alive, s, 0.0), alive


def choose(l, k, kind, bias=None, n_group=1, topk_group=1, group_top=2):
    """The k ids of one token, -1 where nothing is left."""
    s, alive = scores(l, kind)
    c = s if bias is None else s + np.asarray(bias, np.float64)
    alive = alive & (c > -np.inf)
    size = len(c) // n_group
    ranked = []
    for g in range(n_group):
        best = sorted((c[e] for e in range(g * size, (g + 1) * size) if alive[e]), reverse=True)
        ranked.append((-(sum(best[:group_top])) if best else np.inf, g))
    kept = {g for _, g in sorted(ranked)[:topk_group]}
    left = [(-c[e], e) for e in range(len(c)) if alive[e] and e // size in kept]
    ids = [e for _, e in sorted(left)[:k]]
    return ids + [-1] * (k - len(ids))


def weigh(l, ids, kind, renormalize=True, scale=1.0):
    """Weights of one token's ids."""
    s, _ = scores(l, kind)
    w = np.array([s[e] if e >= 0 else 0.0 for e in ids])
    if renormalize:
        w = w / w.sum() if w.sum() > 0 else w
    return scale * w


def router(logits, k, kind="sigmoid", bias=None, n_group=1, topk_group=1, group_top=2,
           renormalize=True, scale=1.0):
    ids = np.array([choose(l, k, kind, bias, n_group, topk_group, group_top) for l in logits],
                   dtype=np.int64).reshape(len(logits), k)
    w = np.array([weigh(l, i, kind, renormalize, scale) for l, i in zip(logits, ids)])
    return ids, w.reshape(len(logits), k)


def backward(logits, ids, grad, kind="sigmoid", renormalize=True, scale=1.0):
    """Gradient of sum(grad * weights) with respect to the logits, by the chain
    rule through the scores."""
    out = np.zeros(np.shape(logits))
    for t, (l, row, g) in enumerate(zip(np.asarray(logits, np.float64), ids, grad)):
        s, _ = scores(l, kind)
        ds = np.zeros_like(s)
        taken = [j for j, e in enumerate(row) if e >= 0]
        total = sum(s[row[j]] for j in taken)
        if renormalize and not total > 0:
            continue
        mean = sum(g[j] * s[row[j]] for j in taken) / total if renormalize else 0.0
        for j in taken:
            ds[row[j]] += scale * ((g[j] - mean) / total if renormalize else g[j])
        out[t] = ds * s * (1 - s) if kind == "sigmoid" else s * (ds - (ds * s).sum())
    return out
