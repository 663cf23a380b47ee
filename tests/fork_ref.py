"""Plain models of the pages that several sequences hold and of the
verification of drafts, on the host.  They share no code with the library."""
from __future__ import annotations

import math

import numpy as np


def up(n, page):
    return -(-n // page)


class Pages:
    """ref, and rows (table, held, lens) as lists; `bad`: a call met something
    outside the table or the pages."""

    def __init__(self, pages, width, page):
        self.ref = [0] * pages
        self.width, self.page, self.bad = width, page, False

    def _good(self, p):
        return 0 <= p < len(self.ref)

    def fork(self, rows, source):
        out = []
        for b in source:
            if b < 0 or b >= len(rows) or rows[b][2] < 0:
                self.bad |= b >= len(rows)
                out.append(([-1] * self.width, 0, -1))
                continue
            table, held, n = rows[b]
            want = up(n, self.page)
            self.bad |= want > held
            cols = min(want, held)
            new = []
            for p in table[:cols]:
                if self._good(p):
                    self.ref[p] += 1
                else:
                    p, self.bad = -1, True
                new.append(p)
            out.append((new + [-1] * (self.width - cols), cols, n))
        return out

    def trim(self, rows, lens=None):
        for b, (table, held, _) in enumerate(rows):
            n = -1 if lens is None else lens[b]
            keep = min(held, up(n, self.page) if n >= 0 else 0)
            for c in range(keep, held):
                p, table[c] = table[c], -1
                if self._good(p) and self.ref[p] > 0:
                    self.ref[p] -= 1
                else:
                    self.bad = True
            rows[b] = (table, keep, rows[b][2])

    def reserve(self, rows, T, count=None):
        B, page = len(rows), self.page
        asks = {}
        for b, (table, held, n) in enumerate(rows):
            c = T if count is None else count[b]
            if n < 0:
                continue
            self.bad |= c > T
            c = min(c, T)
            if c <= 0:
                continue
            first, last = n // page, up(n + c, page)
            good = last <= self.width and up(n, page) <= held
            for col in range(first, min(held, last)) if good else ():
                p = table[col]
                r = self.ref[p] if self._good(p) else 0
                good = good and r >= 1 and (r == 1 or col == first)
            if good:
                asks[b] = (c, first, last)
            else:
                self.bad = True
        # who writes into a page that others hold
        by_page = {}
        for b, (c, first, last) in asks.items():
            if first < rows[b][1] and self.ref[rows[b][0][first]] > 1:
                by_page.setdefault(rows[b][0][first], []).append(b)
        leaves = set()
        for p, who in by_page.items():
            leaves |= set(who if len(who) < self.ref[p] else who[:-1])
        need = {b: (b in leaves) + max(0, last - rows[b][1]) for b, (c, first, last) in asks.items()}
        free = [p for p, r in enumerate(self.ref) if r == 0]
        granted, src, dst = [0] * B, [-1] * B, [-1] * B
        if sum(need.values()) > len(free):
            self.bad = True
            return granted, src, dst
        take = iter(free)
        for b in sorted(asks):
            c, first, last = asks[b]
            table, held, n = rows[b]
            if b in leaves:
                old, new = table[first], next(take)
                self.ref[old] -= 1
                self.ref[new] = 1
                table[first] = new
                if n % page:
                    src[b], dst[b] = old, new
            for col in range(held, last):
                table[col] = next(take)
                self.ref[table[col]] = 1
            rows[b] = (table, max(held, last), n)
            granted[b] = c
        return granted, src, dst


def verify(p, q, tokens, parent, count, u):
    """One sequence: p, q [T, V] float64 (q None: chosen drafts).  Returns
    (path, token, margin): margin is how near (relative to the sums) the
    nearest decision came to its border."""
    T, V = p.shape
    node, path, margin = 0, [0], 1.0
    rest, total = p[0].copy(), 1.0
    scale = 0.0
    t = 0
    while True:
        drafts = [i for i in range(max(t, node) + 1, count)
                  if (i - 1 if parent is None else parent[i]) == node and 0 <= tokens[i] < V]
        if not drafts:
            break
        t = drafts[0]
        x = int(tokens[t])
        left = u[t] * (q[node, x] if q is not None else 1.0) * total
        margin = min(margin, abs(left - rest[x]) / max(left, rest[x]) if max(left, rest[x]) > 0 else 1.0)
        if left < rest[x]:
            node = t
            path.append(t)
            rest, total, scale = p[node].copy(), 1.0, 0.0
            continue
        if q is not None:
            scale += total
            rest = np.maximum(p[node] - scale * q[node], 0.0)
        else:
            rest[x] = 0.0
        total = math.fsum(rest)
    if not math.fsum(rest) > 0.0:
        rest = p[node]
    total = math.fsum(rest)
    if not (0.0 < total < math.inf):
        return path, -1, margin
    target = u[0] * total
    upto = np.cumsum(rest)
    some = np.flatnonzero(rest > 0)
    past = np.flatnonzero((upto > target) & (rest > 0))
    token = int(past[0]) if len(past) else int(some[-1])
    margin = min(margin, float(np.abs(upto[some] - target).min()) / total) if u[0] > 0 else margin
    return path, token, margin
