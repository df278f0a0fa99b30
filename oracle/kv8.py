"""A cache held in 8 bits and attention over it, in binary64 on host arrays: the
definition of ss_rotate and of the ss_cache calls on scaled caches."""
from __future__ import annotations

import numpy as np

from oracle.cache import Pages

X_MIN, X_MAX = -60, 60


def decode(b):
    """What bytes of 1 sign, 4 exponent and 3 mantissa bits stand for."""
    b = np.asarray(b).astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b & 128, -v, v)


def encode(x):
    """The nearest of them, ties to even; beyond 448 the largest, what is not finite a NaN."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.where(np.isfinite(x), np.abs(x), 0.0), 448.0)
    _, e = np.frexp(a)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    a = np.rint(a / step) * step
    _, e = np.frexp(a)
    e = np.where(a > 0, np.maximum(e - 1, -7), -7)  # -7: below the least normal number
    bits = np.where(e < -6, a * 2.0 ** 9, (e + 7) * 8 + np.rint(a / np.exp2(e.astype(float)) * 8) - 8)
    bits = np.where(np.isfinite(x), bits, 127).astype(np.uint8)
    return bits | (np.signbit(x).astype(np.uint8) << 7)


def exponent(amax):
    """The least whole x with amax <= 448 2^x, within the scale's range."""
    m, e = np.frexp(amax)
    x = e - 9 + (m > 0.875)
    return int(min(max(x, X_MIN), X_MAX)) if amax > 0 else X_MIN


def turn(x, pos, inv_freq, magnitude, interleaved):
    """x [..., heads, dim] by positions [...]: pairs times complex numbers."""
    f = np.asarray(inv_freq, np.float64)
    n = len(f)
    w = magnitude * np.exp(1j * (np.asarray(pos, np.float64)[..., None] * f))[..., None, :]
    x = np.array(x, np.float64)
    lo, hi = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else \
        (slice(0, n), slice(n, 2 * n))
    z = (x[..., lo] + 1j * x[..., hi]) * w
    x[..., lo], x[..., hi] = z.real, z.imag
    return x


def above(parents):
    """[N, N]: whether node j is node n or above it; no row for nodes below no root."""
    N = len(parents)
    sees = np.zeros((N, N), bool)
    sees[0, 0] = True
    for n in range(1, N):
        if 0 <= parents[n] < n and sees[parents[n], parents[n]]:
            sees[n] = sees[parents[n]]
            sees[n, n] = True
    return sees


def depths(parents):
    """Edges up to the root, or to the node that hangs below none."""
    d = [0] * len(parents)
    for n in range(1, len(parents)):
        if 0 <= parents[n] < n:
            d[n] = d[parents[n]] + 1
    return d


class Pages8(Pages):
    """pool: bytes [planes, pages, page, heads, dim]; scales: [planes, pages, blocks, heads]."""

    def __init__(self, pool, scales, rows, max_blocks):
        super().__init__(pool, rows, max_blocks)
        self.scales = scales
        self.block = self.ps // scales.shape[2]

    def _carry(self, new, old, slots):
        super()._carry(new, old, slots)
        n = -(-slots // self.block)
        self.scales[:, new, :n] = self.scales[:, old, :n]

    def _copy(self, dst, src):
        super()._copy(dst, src)
        self.scales[:, dst] = self.scales[:, src]

    def _shift(self, b, by):
        """Bytes rounded again under a scale that is 2^-by times the old one."""
        return np.where(by < 0, encode(decode(b) * np.exp2(by)), b)

    def _move(self, moves):
        """A block's scale becomes the largest that its kept slots had."""
        scales, pool = self.scales.copy(), self.pool.copy()
        by_block = {}
        for sp, s, dp, d in moves:
            by_block.setdefault((dp, d // self.block), []).append((sp, s, d))
        for (dp, i), group in by_block.items():
            first = group[0][2]
            own = scales[:, dp, i].astype(int)
            most = np.zeros_like(own) if first % self.block == 0 else own.copy()
            for sp, s, _ in group:
                most = np.maximum(most, scales[:, sp, s // self.block])
            for d in range(i * self.block, first):
                self.pool[:, dp, d] = self._shift(pool[:, dp, d], (own - most)[:, :, None])
            for sp, s, d in group:
                was = scales[:, sp, s // self.block].astype(int)
                self.pool[:, dp, d] = self._shift(pool[:, sp, s], (was - most)[:, :, None])
            self.scales[:, dp, i] = most

    def tokens(self, N, base=None, counts=None, reserved=None):
        """Row by row the base and the tokens of a step."""
        out = []
        for b, at in enumerate(self.lens if base is None else base):
            n = N if counts is None else min(max(counts[b], 0), N)
            if at < 0 or at > self.M * self.ps or (reserved is not None and not reserved[b]):
                at, n = 0, 0
            out.append((at, n))
        return out

    def write(self, plane, x, B, base=None, counts=None, reserved=None):
        """x [B, N, heads, dim] into the slots behind base."""
        for b, (at, n) in enumerate(self.tokens(x.shape[1], base, counts, reserved)[:B]):
            s = at
            while s < at + n:
                end = min(at + n, (s // self.block + 1) * self.block)
                new, first = x[b, s - at:end - at], s
                s = end
                if first // self.ps >= self.M:
                    break
                page = self.tables[b][first // self.ps]
                if not self.held(page) or self.ref[page] > 1:
                    continue
                i, f = first % self.ps // self.block, first % self.block
                for h in range(x.shape[2]):
                    v = np.abs(new[:, h])
                    e = exponent(np.max(np.where(np.isfinite(v), v, 0.0)))
                    at0 = i * self.block
                    if f:
                        was = int(self.scales[plane, page, i, h]) - 127
                        e = max(e, was)
                        held = self.pool[plane, page, at0:at0 + f, h]
                        self.pool[plane, page, at0:at0 + f, h] = self._shift(held, was - e)
                    self.pool[plane, page, at0 + f:at0 + f + len(new), h] = encode(new[:, h] * 2.0 ** -e)
                    self.scales[plane, page, i, h] = e + 127

    def read(self, plane, b, start, N):
        """Slots start .. start + N - 1 of row b, 0 where there is none."""
        out = np.zeros((N, *self.pool.shape[3:]))
        for i in range(N):
            s = start + i
            if 0 <= s < self.M * self.ps and self.held(self.tables[b][s // self.ps]):
                page, at = self.tables[b][s // self.ps], s % self.ps
                x = self.scales[plane, page, at // self.block].astype(float) - 127
                out[i] = decode(self.pool[plane, page, at]) * np.exp2(x)[:, None]
        return out

    def attend(self, q, scale, base=None, counts=None, parents=None, reserved=None, k_plane=0,
               v_plane=1):
        """q [B, N, q_heads, dim]. Returns the result, the logarithms of the sums, and for
        tolerances: the sum of weights times |v|, the largest sum of |q k|, and the largest
        weight times its value's scale, times the sum of the values without theirs."""
        B, N, H, D = q.shape
        out, size, least = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
        lse, dots = np.full((B, N, H), -np.inf), np.zeros((B, N, H))
        for b, (at, n) in enumerate(self.tokens(N, base, counts, reserved)[:B]):
            end = min(at + n, self.M * self.ps)
            if not n or not end:
                continue
            k, v = self.read(k_plane, b, 0, end), self.read(v_plane, b, 0, end)
            x = np.array([self.scales[v_plane, self.tables[b][s // self.ps], s % self.ps // self.block]
                          if self.held(self.tables[b][s // self.ps]) else v[0, :, 0] * 0 + 127
                          for s in range(end)])
            x = np.exp2(x - 127.0)
            there = np.array([self.held(self.tables[b][s // self.ps]) for s in range(end)])
            for t in range(n):
                sees = there.copy()
                if parents is None:
                    sees[at + t + 1:] = False
                else:
                    up = above(parents[b])[t]
                    if not up.any():
                        continue
                    sees[at:] &= up[:max(end - at, 0)]
                if not sees.any():
                    continue
                for h in range(H):
                    c = h // (H // k.shape[1])
                    s = k[sees, c] @ q[b, t, h] * scale
                    m = s.max()
                    with np.errstate(invalid="ignore"):
                        w = np.exp(s - m)
                    out[b, t, h] = w @ v[sees, c] / w.sum()
                    size[b, t, h] = w @ np.abs(v[sees, c]) / w.sum()
                    least[b, t, h] = (w * x[sees, c]).max() / w.sum() * \
                        (np.abs(v[sees, c]) / x[sees, c][:, None]).sum(0)
                    lse[b, t, h] = m + np.log(w.sum())
                    dots[b, t, h] = (np.abs(k[sees, c]) @ np.abs(q[b, t, h])).max() * scale
        return out, lse, size, dots, least
