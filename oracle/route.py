"""Routing of tokens to experts and its gradient, one token after another in 64 bits."""

from __future__ import annotations

import numpy as np

NEVER = -np.inf


def scores(x, score):
    """softmax or sigmoid of a token's logits; -inf (and NaN) count as absent."""
    x = np.asarray(x, np.float64)
    there = x > NEVER
    s = np.zeros_like(x)
    if score == "softmax":
        if there.any():
            e = np.exp(x[there] - x[there].max())
            s[there] = e / e.sum()
    else:
        s[there] = 1 / (1 + np.exp(-x[there]))
    return s


def best(values, count):
    """The `count` largest, in descending order, ties to the lowest place."""
    return sorted(range(len(values)), key=lambda i: (-values[i], i))[:count]


def route_token(x, k, score="softmax", bias=None, groups=1, top_groups=1, renorm=False, scale=1.0):
    """(indices, weights, margin): margin is the smallest difference of two
    values that the choice told apart."""
    x = np.asarray(x, np.float64)
    E = len(x)
    s = scores(x, score)
    c = np.where(x > NEVER, x if bias is None and groups == 1 else s + (0 if bias is None else bias), NEVER)
    gaps = []
    if groups > 1:
        size = E // groups
        worth = [sum(sorted(c[g * size:(g + 1) * size])[::-1][:2]) for g in range(groups)]
        stay = best(worth, groups)
        gaps += [worth[a] - worth[b] for a, b in zip(stay[:top_groups], stay[1:]) if worth[b] > NEVER]
        for g in stay[top_groups:]:
            c[g * size:(g + 1) * size] = NEVER
    order = best(c, min(k + 1, E))
    gaps += [c[a] - c[b] for a, b in zip(order, order[1:]) if c[b] > NEVER]
    index = [i if c[i] > NEVER else -1 for i in order[:k]] + [-1] * (k - len(order[:k]))
    w = np.array([s[i] if i >= 0 else 0.0 for i in index])
    if renorm:
        w = w / w.sum() if w.sum() > 0 else w * 0
    gaps = [g for g in gaps if g != 0]                # exact ties are decided by the place
    return index, w * scale, min(gaps, default=np.inf)


def weights_at(x, index, score, renorm, scale):
    """The weights of a fixed choice, as a function of the logits."""
    s = scores(x, score)
    w = np.array([s[i] if i >= 0 else 0.0 for i in index])
    if renorm and w.sum() > 0:
        w = w / w.sum()
    return w * scale


def backward_token(x, index, grad, score, renorm, scale):
    """d (grad . weights) / d x: the chain rule over the full Jacobians."""
    x = np.asarray(x, np.float64)
    E, k = len(x), len(index)
    s = scores(x, score)
    ds = np.diag(s) - np.outer(s, s) if score == "softmax" else np.diag(s * (1 - s))     # [of score, by logit]
    pick = np.zeros((k, E))
    for r, i in enumerate(index):
        if i >= 0:
            pick[r, i] = 1.0
    u = pick @ s
    dw = np.eye(k)
    if renorm:
        dw = np.eye(k) / u.sum() - np.outer(u, np.ones(k)) / u.sum() ** 2 if u.sum() > 0 else np.zeros((k, k))
    return np.asarray(grad, np.float64) @ (scale * dw @ pick @ ds)
