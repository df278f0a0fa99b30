"""Pages of a key/value cache on host lists: the definition of the ss_cache calls."""
from __future__ import annotations

import numpy as np


class Pages:
    """pool: [planes, pages, page, heads, dim]; tables / ref / lens: plain lists."""

    def __init__(self, pool, rows, max_blocks):
        self.pool = pool
        self.P, self.ps = pool.shape[1], pool.shape[2]
        self.tables = [[-1] * max_blocks for _ in range(rows)]
        self.ref = [0] * self.P
        self.lens = [0] * rows
        self.M = max_blocks

    def held(self, page):
        return 0 <= page < self.P

    def pages_of(self, slots):
        return -(-slots // self.ps)

    def _drop(self, row, first):
        for i in range(first, self.M):
            if self.held(self.tables[row][i]):
                self.ref[self.tables[row][i]] -= 1
            self.tables[row][i] = -1

    def _carry(self, new, old, slots):
        self.pool[:, new, :slots] = self.pool[:, old, :slots]

    def _move(self, moves):
        for sp, s, dp, d in moves:
            self.pool[:, dp, d] = self.pool[:, sp, s]

    def _copy(self, dst, src):
        self.pool[:, dst] = self.pool[:, src]

    def reserve(self, add, base=None):
        base = list(self.lens if base is None else base)
        before = list(self.ref)
        free = [p for p in range(self.P) if before[p] == 0]
        ok, used = [], 0
        for b, n in enumerate(add):
            if base[b] < 0 or n < 0 or (n > 0 and base[b] + n > self.M * self.ps):
                ok.append(0)
                continue
            lo, hi = base[b] // self.ps, self.pages_of(base[b] + n)
            tab = self.tables[b]
            need = [i for i in range(lo, hi) if n > 0 and
                    (not self.held(tab[i]) or before[tab[i]] > 1)]
            first, used = used, used + len(need)
            ok.append(int(used <= len(free)))
            if not ok[-1]:
                continue
            for k, i in enumerate(need):
                new, old = free[first + k], tab[i]
                if self.held(old):
                    self.ref[old] -= 1
                    if i == lo:
                        self._carry(new, old, base[b] % self.ps)
                self.ref[new] += 1
                tab[i] = new
        return ok

    def fork(self, src, dst):
        R = len(self.tables)
        ok = []
        for i, (s, d) in enumerate(zip(src, dst)):
            ok.append(int(0 <= s < R and 0 <= d < R and d not in src and list(dst).count(d) == 1))
        tables, lens = [list(t) for t in self.tables], list(self.lens)
        for s, d, good in zip(src, dst, ok):
            if good:
                self._drop(d, 0)
                for i in range(min(self.M, self.pages_of(max(lens[s], 0)))):
                    if self.held(tables[s][i]):
                        self.tables[d][i] = tables[s][i]
                        self.ref[tables[s][i]] += 1
                self.lens[d] = lens[s]
        return ok

    def commit(self, acc, nodes=None, base=None, release=True, reserved=None):
        base = list(self.lens if base is None else base)
        before = list(self.ref)
        room = self.M * self.ps
        ok = []

        def own(page):
            return self.held(page) and before[page] <= 1

        for b, n in enumerate(acc):
            good = base[b] >= 0 and n >= 0 and base[b] + 1 + n <= room
            good = good and (reserved is None or reserved[b] != 0)
            good = good and all(own(self.tables[b][i])
                                for i in range(base[b] // self.ps, self.pages_of(base[b] + 1 + n)))
            moves = []
            if good and nodes is not None:
                N = len(nodes[b])
                good = n < N
                prev = 0
                for i in range(n if good else 0):
                    node = int(nodes[b][i])
                    good = good and prev < node < N and base[b] + node < room
                    prev = node
                    if good and node != i + 1:
                        s, d = base[b] + node, base[b] + 1 + i
                        sp, dp = self.tables[b][s // self.ps], self.tables[b][d // self.ps]
                        good = own(sp) and own(dp)
                        moves.append((sp, s % self.ps, dp, d % self.ps))
            ok.append(int(good))
            if not good:
                continue
            self._move(moves)
            self.lens[b] = base[b] + 1 + n
            if release:
                self._drop(b, self.pages_of(self.lens[b]))
        return ok

    def truncate(self, new_len=None, rows=None):
        n = len(rows) if rows is not None else len(new_len) if new_len is not None else len(self.lens)
        for i in range(n):
            row = i if rows is None else rows[i]
            keep = 0 if new_len is None else max(new_len[i], 0)
            if 0 <= row < len(self.lens):
                self._drop(row, self.pages_of(keep))
                self.lens[row] = min(self.lens[row], keep)

    def copy_pages(self, src, dst):
        ok = [int(self.held(s) and self.held(d) and d not in src and list(dst).count(d) == 1)
              for s, d in zip(src, dst)]
        for s, d, good in zip(src, dst, ok):
            if good:
                self._copy(d, s)
        return ok

    def consistent(self):
        """Every count is the number of table entries that name the page."""
        n = np.bincount([p for t in self.tables for p in t if self.held(p)], minlength=self.P)
        return n.tolist() == self.ref
