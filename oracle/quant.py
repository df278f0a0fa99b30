"""LM-head logits of 4-bit weights with group scales, binary64."""
from __future__ import annotations

import numpy as np


def unpack(q):
    """[..., n] bytes -> [..., 2 n] nibbles, the low one first."""
    return np.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], -1)


def weights(qweight, scales, zeros, group):
    """The weights [V, K] in binary64 (exact: 4-bit integers times 16-bit scales)."""
    n = unpack(qweight).astype(np.float64)
    K = n.shape[1]
    g = np.arange(K) // group
    z = 8.0 if zeros is None else unpack(zeros).astype(np.float64)[:, g]
    return (n - z) * scales.astype(np.float64)[:, g]


def logits(hidden, qweight, scales, zeros, group):
    return hidden.astype(np.float64) @ weights(qweight, scales, zeros, group).T


def error_bound(hidden, scales, group):
    """What a sum in binary32 may be off, per logit. A group's sum has at most
    group + 1 terms (16 + n) x and (16 + z) sum x, all at most 31 |x| in size, so
    every partial sum is at most 62 S, S the group's sum of |x|; each of its
    group + 1 additions, and the group + 1 roundings of sum x and its product
    (31 S each), is off by at most one step, 2^-23 of that. Scaling and adding
    groups rounds two times per group more, on sums of at most 62 sum |s| S."""
    B, K = hidden.shape
    G = scales.shape[1]
    x = np.zeros((B, G * group))
    x[:, :K] = np.abs(hidden.astype(np.float64))
    S = x.reshape(B, G, group).sum(-1)
    mass = S @ np.abs(scales.astype(np.float64)).T
    return 2.0 ** -23 * 62 * (2 * (group + 1) + 2 * G) * mass
