"""Plain references of the paged KV cache's operators: attention in 64 bits,
position by position as defined, and the pages' life as a sequential program."""
from __future__ import annotations

import numpy as np

BF16_HALF = 2.0 ** -8      # a BF16 rounding, relative to the value
F32_HALF = 2.0 ** -24


def places(lens, cu):
    """(row, position) of every token below cu[-1]."""
    return [(s, int(lens[s]) - (int(cu[s + 1]) - int(cu[s])) + i)
            for s in range(len(lens)) for i in range(int(cu[s + 1]) - int(cu[s]))]


def sees(p, t, window, sinks):
    return t <= p and (window == 0 or t > p - window or t < sinks)


def attention(q, keys, values, lens, cu, scale, window=0, sinks=0):
    """q [tokens][hq][d] float64; keys[s], values[s] [len][hkv][d] float64 (the
    values that the cache stands for). Returns (out, spread, score error) per
    (token, head): out [tokens][hq][d], sum_t w_t |v_t| of the same shape, and
    the FP32 error of the largest score, as a relative error of a weight:
    (d + 2) roundings of sum |q k| scale, twice (the weight and the sum)."""
    n, hq, d = q.shape
    out, spread, serr = np.zeros((n, hq, d)), np.zeros((n, hq, d)), np.zeros((n, hq, 1))
    for i, (s, p) in enumerate(places(lens, cu)):
        seen = [t for t in range(int(lens[s])) if sees(p, t, window, sinks)]
        if not seen:
            continue
        k, v = keys[s][seen], values[s][seen]
        g = hq // k.shape[1]
        for a in range(hq):
            x = k[:, a // g] @ q[i, a] * scale
            w = np.exp(x - x.max())
            w /= w.sum()
            out[i, a] = w @ v[:, a // g]
            spread[i, a] = w @ np.abs(v[:, a // g])
            serr[i, a] = 2 * (d + 2) * F32_HALF * (np.abs(k[:, a // g]) @ np.abs(q[i, a])).max() * abs(scale)
    return out, spread, serr


class Pages:
    """resize, fork, trim and compact, one row and one page at a time."""

    def __init__(self, n_pages, n_seqs, width, page):
        self.refs = [0] * n_pages
        self.tables = [[-1] * width for _ in range(n_seqs)]
        self.lens = [0] * n_seqs
        self.page, self.width = page, width
        self.copies = []           # (source, target, positions) of the last call

    def _drop(self, s, j):
        if self.tables[s][j] >= 0:
            self.refs[self.tables[s][j]] -= 1
        self.tables[s][j] = -1

    def resize(self, new):
        """False: too few pages (rows that shrink have shrunk)."""
        ps = self.page
        self.copies = []
        for s, n in enumerate(new):
            if 0 <= n < self.lens[s]:
                for j in range(-(-n // ps), self.width):
                    self._drop(s, j)
                self.lens[s] = n
        grow = [(s, n) for s, n in enumerate(new) if n > self.lens[s] and n <= self.width * ps]
        write = [(s, j) for s, n in grow for j in range(self.lens[s] // ps, -(-n // ps))]
        holders = {}
        for s, j in write:
            page = self.tables[s][j]
            if page >= 0 and self.refs[page] > 1:
                holders.setdefault(page, []).append(s)
        keeper = {page: rows[0] for page, rows in holders.items() if len(rows) == self.refs[page]}
        want = [(s, j) for s, j in write if self.tables[s][j] < 0 or
                (self.tables[s][j] in holders and keeper.get(self.tables[s][j]) != s)]
        free = [p for p, r in enumerate(self.refs) if r == 0]
        if len(want) > len(free):
            return False
        for (s, j), fresh in zip(want, free):
            old = self.tables[s][j]
            if old >= 0:
                self.refs[old] -= 1
                if j * ps < self.lens[s]:
                    self.copies.append((old, fresh))
            self.tables[s][j] = fresh
            self.refs[fresh] = 1
        for s, n in grow:
            self.lens[s] = n
        return True

    def fork(self, src):
        """False: some row's fork was not allowed (and not done)."""
        ok = True
        for s, f in enumerate(src):
            if f < 0:
                continue
            if f >= len(src) or f == s or src[f] >= 0 or self.lens[s] or any(x >= 0 for x in self.tables[s]):
                ok = False
                continue
            for j in range(-(-self.lens[f] // self.page)):
                page = self.tables[f][j]
                self.tables[s][j] = page
                if page >= 0:
                    self.refs[page] += 1
            self.lens[s] = self.lens[f]
        return ok

    def trim(self, window, sinks):
        for s in range(len(self.lens)):
            for j in range(self.width):
                positions = range(j * self.page, (j + 1) * self.page)
                if not any(t < sinks or t > self.lens[s] - window for t in positions):   # for p = len, and every later p
                    self._drop(s, j)

    def compact(self):
        self.copies = []
        n = sum(r > 0 for r in self.refs)
        holes = [p for p in range(n) if self.refs[p] == 0]
        movers = [p for p in range(n, len(self.refs)) if self.refs[p] > 0]
        to = dict(zip(movers, holes))
        for m, h in to.items():
            self.refs[h], self.refs[m] = self.refs[m], 0
            self.copies.append((m, h))
        self.tables = [[to.get(x, x) for x in row] for row in self.tables]
