"""Plain definitions of the paged cache's operations for the tests: page
bookkeeping one entry at a time on Python lists, attention and scores in
float64.  Shares no code with the library."""
from __future__ import annotations

import math

import numpy as np


class Pool:
    """Tables, reference counts and lengths, and what each page holds: content[p][i] is whatever was put at position
    i of page p (any value), None where nothing is defined."""

    def __init__(self, n_pages, page, n_seq, max_pages):
        self.n_pages, self.page, self.n_seq, self.max_pages = n_pages, page, n_seq, max_pages
        self.refs = [0] * n_pages
        self.table = [[-1] * max_pages for _ in range(n_seq)]
        self.lens = [-1] * n_seq
        self.content = [[None] * page for _ in range(n_pages)]

    def reserve(self, n_new):
        """False where the call must change nothing."""
        for b, add in enumerate(n_new):
            if self.lens[b] >= 0 and add > 0 and self.lens[b] + add > self.max_pages * self.page:
                return False
        refs, table = list(self.refs), [list(r) for r in self.table]
        free = [p for p, r in enumerate(self.refs) if r == 0]
        copies = []
        for b, add in enumerate(n_new):
            if self.lens[b] < 0 or add <= 0:
                continue
            first, last = self.lens[b] // self.page, (self.lens[b] + add - 1) // self.page
            for c in range(first, last + 1):
                p = table[b][c]
                if p >= 0 and refs[p] == 1:
                    continue
                if not free:
                    return False
                fresh = free.pop(0)
                if p >= 0:
                    refs[p] -= 1
                    copies.append((p, fresh, max(0, min(self.page, self.lens[b] - c * self.page))))
                table[b][c], refs[fresh] = fresh, 1
        self.refs, self.table = refs, table
        for src, dst, rows in copies:
            self.content[dst][:rows] = self.content[src][:rows]
            self.content[dst][rows:] = [None] * (self.page - rows)
        return True

    def _drop(self, b, c):
        if self.table[b][c] >= 0:
            self.refs[self.table[b][c]] -= 1
            self.table[b][c] = -1

    def fork(self, parents, children):
        rows = [list(self.table[p]) for p in parents]
        lens = [self.lens[p] for p in parents]
        for row, n, b in zip(rows, lens, children):
            row = [p if c * self.page < n else -1 for c, p in enumerate(row)]
            for p in row:
                if p >= 0:
                    self.refs[p] += 1
            for c in range(self.max_pages):
                self._drop(b, c)
            self.table[b], self.lens[b] = row, n

    def free(self, seqs, keep_first=0, keep_last=0):
        for b in seqs:
            n = self.lens[b]
            whole = keep_first == 0 and keep_last == 0
            if n < 0 and not whole:
                continue
            for c in range(self.max_pages):
                lo, hi = c * self.page, (c + 1) * self.page
                kept = [i for i in range(lo, min(hi, n)) if i < keep_first or i >= n - keep_last]
                stays = bool(kept) or hi > n  # or it reaches behind the end
                if whole or not stays:
                    self._drop(b, c)
            if whole:
                self.lens[b] = -1

    def compact(self):
        now, low, high = {}, 0, self.n_pages - 1
        while True:
            while low < self.n_pages and self.refs[low]:
                low += 1
            while high >= 0 and not self.refs[high]:
                high -= 1
            if low >= high:
                break
            self.refs[low], self.refs[high], now[high] = self.refs[high], 0, low
            self.content[low], self.content[high] = self.content[high], [None] * self.page
        self.table = [[now.get(p, p) for p in row] for row in self.table]
        return low

    def put(self, b, pos, value):
        self.content[self.table[b][pos // self.page]][pos % self.page] = value


def visible(n, window, sinks):
    return [p for p in range(n) if window == 0 or p >= n - window or p < sinks]


def attention(q, k, v, scale):
    """One query row of one head over the visible rows k, v (float64): out, log2-sum-exp, sum p |v|, and the largest
    scale sum |q k|."""
    if len(k) == 0:
        return np.zeros(q.shape[-1]), -math.inf, np.zeros(q.shape[-1]), 0.0
    z = scale * (k @ q)
    m = z.max()
    e = np.exp(z - m)
    p = e / e.sum()
    return p @ v, (m + math.log(e.sum())) / math.log(2), p @ np.abs(v), float((scale * np.abs(k) @ np.abs(q)).max())
