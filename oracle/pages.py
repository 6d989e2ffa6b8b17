"""CPU ORACLE of the page calls -- TEST INFRASTRUCTURE ONLY. The rules of hs_pages_* one entry at a
time, on numpy arrays: table [requests, max_pages], refs [pages], free (a Python list, top last),
pools (one [pages * page_size, row_bytes] array per layer). Each call returns the flags it raises."""
from __future__ import annotations

import numpy as np

TOKEN, DUP, STATE, SEQLEN, NOPAGE = 1, 2, 4, 32, 256


class Pages:
    def __init__(self, requests, max_pages, pages, page_size, pools):
        self.table = np.full((requests, max_pages), -1, np.int32)
        self.refs = np.zeros(pages, np.int32)
        self.free = list(range(pages - 1, -1, -1))
        self.ps, self.pools = page_size, pools

    def _grant(self, asks, room):
        """asks: (need or None where refused) per entry -> pages per entry, -1 refused."""
        total, got, flags = 0, [], 0
        for need in asks:
            total += need or 0
            if need is None or (need and total > room):
                got.append(-1)
                flags |= 0 if need is None else NOPAGE
            else:
                got.append(need)
        return got, flags

    def _pop(self):
        page = self.free.pop()
        assert self.refs[page] == 0
        self.refs[page] = 1
        return page

    def _up(self, n):
        return -(-int(n) // self.ps)

    def extend(self, requests, old, new):
        R, most = self.table.shape[0], self.table.shape[1] * self.ps
        asks, flags = [], 0
        for r, a, b in zip(requests, old, new):
            f = 0
            if r < 0:
                asks.append(0)
                continue
            if r >= R:
                f = TOKEN
            elif list(requests).count(r) > 1:
                f = DUP
            elif a < 0 or b < a or b > most:
                f = SEQLEN
            elif (self.table[r, self._up(a):self._up(b)] != -1).any():
                f = STATE
            flags |= f
            asks.append(None if f else self._up(b) - self._up(a))
        got, f = self._grant(asks, len(self.free))
        for r, a, w in zip(requests, old, got):
            for i in range(max(w, 0)):
                self.table[r, self._up(a) + i] = self._pop()
        return got, flags | f

    def fork(self, parents, children, lens):
        R, most = self.table.shape[0], self.table.shape[1] * self.ps
        named = [c for p, c in zip(parents, children) if p >= 0 and c >= 0]
        heads = {p for p, c in zip(parents, children) if p >= 0 and c >= 0}
        asks, flags, pad = [], 0, []
        for p, c, n in zip(parents, children, lens):
            f, need = 0, 0
            pad.append(p < 0 or c < 0)
            if not pad[-1]:
                if p >= R or c >= R:
                    f = TOKEN
                elif named.count(c) > 1 or c in heads:
                    f = DUP
                elif n < 0 or n > most:
                    f = SEQLEN
                elif (self.table[c] != -1).any():
                    f = STATE
                elif n % self.ps:
                    need = int(self.table[p, n // self.ps] >= 0)
            flags |= f
            asks.append(None if f else need)
        got, f = self._grant(asks, len(self.free))
        for p, c, n, w, skip in zip(parents, children, lens, got, pad):
            if skip or w < 0:
                continue
            full, rest = n // self.ps, n % self.ps
            self.table[c, :full] = self.table[p, :full]
            for page in self.table[p, :full]:
                if page >= 0:
                    self.refs[page] += 1
            if w:
                to, src = self._pop(), self.table[p, full]
                self.table[c, full] = to
                for pool in self.pools:
                    pool[to * self.ps:to * self.ps + rest] = pool[src * self.ps:src * self.ps + rest]
        return got, flags | f

    def release(self, requests, first=None, end=None):
        flags, gone = 0, set()
        for i, r in enumerate(requests):
            if r < 0:
                continue
            if r >= self.table.shape[0]:
                flags |= TOKEN
                continue
            lo = max(0, first[i]) if first is not None else 0
            hi = min(self.table.shape[1], end[i]) if end is not None else self.table.shape[1]
            for k in range(lo, hi):
                page = self.table[r, k]
                if page >= 0:
                    self.table[r, k] = -1
                    self.refs[page] -= 1
                    if self.refs[page] == 0:
                        gone.add(int(page))
        self.free += sorted(gone, reverse=True)
        return flags

    def compact(self):
        n = self.refs.size
        live = int((self.refs > 0).sum())
        movers = [p for p in range(live, n) if self.refs[p] > 0]
        holes = [p for p in range(live) if self.refs[p] == 0]
        for m, h in zip(movers, holes):
            self.refs[h], self.refs[m] = self.refs[m], 0
            self.table[self.table == m] = h
            for pool in self.pools:
                pool[h * self.ps:(h + 1) * self.ps] = pool[m * self.ps:(m + 1) * self.ps]
        self.free = list(range(n - 1, live - 1, -1))

    def check(self):
        """Every page is on the stack or held exactly as often as it is counted."""
        held = np.bincount(self.table[self.table >= 0], minlength=self.refs.size)
        assert np.array_equal(held, self.refs)
        assert sorted(self.free) == np.flatnonzero(self.refs == 0).tolist()
