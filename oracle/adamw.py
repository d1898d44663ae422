"""AdamW over one tensor and the gradient norm, from their formulas in 64 bits.

Formulas, with the clipped gradient ``g' = c g``, ``c = min(1, max_norm / (norm + 1e-6))``::

    m' = beta1 m + (1 - beta1) g'
    v' = beta2 v + (1 - beta2) g'^2
    w' = w - lr (m' / (1 - beta1^t) / (sqrt(v' / (1 - beta2^t)) + eps) + wd w)

8-bit moments: per block of 256 elements a scale (largest magnitude over the
format's largest value) and numbers of the format, rounded up with the
probability of the rest, from 16 given random bits.
"""

from __future__ import annotations

import numpy as np

BLOCK = 256
F64 = np.float64


def clip_factor(norm: float, max_norm: float) -> float:
    return min(1.0, max_norm / (float(norm) + 1e-6)) if max_norm > 0 else 1.0


def adamw(w, g, m, v, t, lr, beta1, beta2, eps, wd, clip=1.0):
    """(w', m', v') of step t."""
    w, g, m, v = (np.asarray(x, F64) for x in (w, g, m, v))
    g = g * clip
    m1 = beta1 * m + (1 - beta1) * g
    v1 = beta2 * v + (1 - beta2) * g * g
    update = m1 / (1 - beta1 ** t) / (np.sqrt(v1 / (1 - beta2 ** t)) + eps)
    return w - lr * (update + wd * w), m1, v1


def grad_norm(grads) -> float:
    return float(np.sqrt(sum(np.dot(np.asarray(g, F64), np.asarray(g, F64)) for g in grads)))


def random_bits(seed: int, block, place):
    """The 32 bits that round the element at `place` of block `block`."""
    def mix(x):
        x = x ^ (x >> 16)
        x = x * 0x6A09E667 % 2 ** 32
        x = x ^ (x >> 15)
        x = x * 0xBB67AE85 % 2 ** 32
        return x ^ (x >> 16)
    block, place = np.asarray(block, np.uint64), np.asarray(place, np.uint64)
    key = mix((mix(block % 2 ** 32 ^ np.uint64(seed % 2 ** 32)) + np.uint64(seed >> 32)) % 2 ** 32)
    return mix((key + place * 0x9E3779B9) % 2 ** 32)


def spacing(y, mantissa, least):
    """Distance of the format's numbers at y >= 0."""
    e = np.frexp(y)[1] - 1
    return np.exp2(np.maximum(e, least) - mantissa)


E4M3 = dict(top=448.0, mantissa=3, least=-6)
E5M2 = dict(top=57344.0, mantissa=2, least=-14)


def encode(x, r16, top, mantissa, least):
    """(numbers, scales, unrounded position in spacings) of one tensor's
    values x: numbers * scale stands for x."""
    x = np.asarray(x, F64)
    n = x.size
    pad = np.zeros(-(-n // BLOCK) * BLOCK)
    pad[:n] = np.abs(x)
    scale = pad.reshape(-1, BLOCK).max(1) / top
    per = np.repeat(scale, BLOCK)[:n]
    y = np.divide(np.abs(x), per, out=np.zeros(n), where=per > 0)
    q = spacing(y, mantissa, least)
    at = y / q + np.asarray(r16, F64) / 65536
    return np.copysign(np.minimum(np.floor(at) * q, top), x), scale, at
