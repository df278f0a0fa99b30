"""Verification of drafts against probability rows with given uniforms, binary64."""
from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np


@dataclass
class Verified:
    tokens: list      # accepted drafts, then the final token
    n_acc: int
    margin: float     # distance of the final draw to the nearest running sum, over the whole sum


def pick(r, u):
    """Lowest v whose running sum exceeds u times the whole sum (-1: no mass); for
    u outside [0, 1) the last entry with mass. Sums are binary64."""
    r = np.where(r > 0, r, 0.0)  # negative and NaN entries hold no mass
    cum = np.cumsum(r)
    total = cum[-1]
    if not total > 0:
        return -1, math.inf
    hit = np.nonzero((cum > u * total) & (r > 0))[0]
    if hit.size == 0:
        return int(np.nonzero(r > 0)[0][-1]), math.inf
    return int(hit[0]), float(np.min(np.abs(cum / total - u)))


def verify(p, q, drafts, u, n):
    """One request: p [G+1, V], q [G, V] or None, drafts [G], u [G+1], n drafts used."""
    p = np.asarray(p, np.float64)
    V = p.shape[1]
    G = p.shape[0] - 1
    n = min(max(int(n), 0), G)
    out = []
    for j in range(n):
        d = int(drafts[j])
        if 0 <= d < V:
            qd = 1.0 if q is None else float(q[j][d])
            if float(u[j]) * qd < p[j, d]:
                out.append(d)
                continue
        if q is None:
            r = p[j].copy()
            if 0 <= d < V:
                r[d] = 0.0
        else:
            with np.errstate(invalid="ignore"):
                r = p[j] - np.asarray(q[j], np.float64)
        if not np.where(r > 0, r, 0.0).sum() > 0:
            r = p[j]
        t, m = pick(r, float(u[G]))
        return Verified(out + [t], j, m)
    t, m = pick(p[n], float(u[G]))
    return Verified(out + [t], n, m)
