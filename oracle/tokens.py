"""Embedding, layer norm, dropout and token log probabilities with their gradients, in 64 bits from the definitions."""

from __future__ import annotations

import numpy as np

LOW = 0xFFFFFFFF


def embed(table, tokens, scale=1.0):
    table, tokens = np.asarray(table, np.float64), np.asarray(tokens)
    y = np.zeros((*tokens.shape, table.shape[1]))
    there = (tokens >= 0) & (tokens < len(table))
    y[there] = table[tokens[there]] * scale
    return y


def embed_backward(grad, tokens, vocab, scale=1.0, onto=None):
    """(the gradient of the table, the sum of its terms' magnitudes, how many terms each row has)."""
    grad = np.asarray(grad, np.float64).reshape(-1, grad.shape[-1])
    d = np.zeros((vocab, grad.shape[1])) if onto is None else np.array(onto, np.float64)
    size, count = np.abs(d), np.zeros(vocab, np.int64)
    for i, t in enumerate(np.asarray(tokens).reshape(-1)):
        if 0 <= t < vocab:
            d[t] += grad[i] * scale
            size[t] += np.abs(grad[i] * scale)
            count[t] += 1
    return d, size, count


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    x = np.asarray(x, np.float64)
    mean = x.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + eps)
    y = (x - mean) * rstd
    y = y if weight is None else y * np.asarray(weight, np.float64)
    return y if bias is None else y + np.asarray(bias, np.float64), np.concatenate([mean, rstd], -1)


def layer_norm_backward(grad, x, stats, weight=None):
    """(dx, dw, db) by the formula, with the row's statistics as they are given."""
    grad, x, stats = (np.asarray(a, np.float64) for a in (grad, x, stats))
    xh = (x - stats[..., :1]) * stats[..., 1:]
    g = grad if weight is None else grad * np.asarray(weight, np.float64)
    dx = stats[..., 1:] * (g - g.mean(-1, keepdims=True) - xh * (g * xh).mean(-1, keepdims=True))
    rows = tuple(range(x.ndim - 1))
    return dx, (grad * xh).sum(rows), grad.sum(rows)


def philox(counter, key):
    """Philox4x32-10 of one block, in whole numbers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & LOW, (a >> 32) ^ c[3] ^ k[1], a & LOW]
        k = [(k[0] + 0x9E3779B9) & LOW, (k[1] + 0xBB67AE85) & LOW]
    return c


def random_bits(element, seed, offset):
    """The 32 bits that decide over an element."""
    key = (seed & LOW, seed >> 32)
    halves = []
    for which in (0, 1):
        word = philox((element >> 3 & LOW, element >> 35, offset & LOW, offset >> 32 | which << 31), key)[element % 8 // 2]
        halves.append(word >> 16 if element % 2 else word & 0xFFFF)
    return halves[0] << 16 | halves[1]


def drop(x, p, seed, offset=0, residual=None):
    x = np.asarray(x, np.float64)
    least = round(p * 2 ** 32)
    keep = np.array([random_bits(e, seed, offset) >= least for e in range(x.size)]).reshape(x.shape)
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(keep, x / (1 - p), 0.0)
    return y if residual is None else y + np.asarray(residual, np.float64)


def logprobs(logits, target=None, top=0, scale=1.0):
    """One row: (logp, entropy, (largest, log of the sum), indices, their log probabilities)."""
    z = np.asarray(logits, np.float64) * scale
    if target is not None and not 0 <= target < len(z):
        return 0.0, 0.0, (0.0, 0.0), [-1] * top, [0.0] * top
    m = np.fmax.reduce(z)
    if not m > -np.inf and not np.isnan(z).any():
        return -np.inf, 0.0, (-np.inf, 0.0), [-1] * top, [-np.inf] * top
    bad = np.isnan(z).any() or m == np.inf
    with np.errstate(invalid="ignore", over="ignore"):
        d = z - m
        total = np.exp(d).sum()
        entropy = np.log(total) - np.where(d > -np.inf, np.exp(d) * np.where(d > -np.inf, d, 0), 0).sum() / total
    order = sorted((i for i in range(len(z)) if z[i] > -np.inf), key=lambda i: (-z[i], i))[:top]
    nan = np.nan
    alternatives = [nan if bad else z[i] - m - np.log(total) for i in order]
    rest = top - len(order)
    return (None if target is None else nan if bad else z[target] - m - np.log(total), nan if bad else entropy,
            (m, nan if bad else np.log(total)), order + [-1] * rest, alternatives + [nan if bad else -np.inf] * rest)


def logprobs_backward(logits, target, grad_logp=0.0, grad_entropy=0.0, scale=1.0):
    """One row, by the chain rule over the full Jacobian of the log probabilities."""
    z = np.asarray(logits, np.float64) * scale
    if target is not None and not 0 <= target < len(z):
        return np.zeros(len(z))
    m = z.max()
    if m == -np.inf:
        return np.zeros(len(z))
    p = np.exp(z - m) / np.exp(z - m).sum()
    logp = np.log(np.where(p > 0, p, 1.0))
    # the Jacobian of log p_i by z_j is [i = j] - p_j; H = -sum p log p
    by = -grad_entropy * p * (1 + logp)
    if target is not None:
        by = by + grad_logp * (np.arange(len(z)) == target)
    return (by - p * by.sum()) * scale
