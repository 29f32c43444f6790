"""The calls on a cache's pages as their definitions say, one entry after another, for their tests (plain Python)."""
from __future__ import annotations


class PoolModel:
    """Page tables, lengths, slots and counts of n_seq sequences."""

    def __init__(self, n_seq, max_pages, page, n_pages, bits):
        self.P, self.n_pages, self.bits = page, n_pages, bits
        self.pages = [[-1] * max_pages for _ in range(n_seq)]
        self.lens, self.slots, self.refs = [0] * n_seq, list(range(n_seq)), [0] * n_pages

    def valid(self, page):
        return 0 <= page < self.n_pages

    def release(self, keep, window=0, sinks=0):
        for row, n in zip(self.pages, keep):
            for b in range(len(row)):
                behind = window > 0 and (b + 1) * self.P <= n - window + 1 and b * self.P >= sinks
                if b * self.P >= n or behind:
                    if self.valid(row[b]):
                        self.refs[row[b]] -= 1
                    row[b] = -1

    def fork(self, parent):
        """slot_src, slot_dst"""
        n = len(parent)
        ok = [p if 0 <= p < n else None for p in parent]
        old_pages, old_lens, old_slots = self.pages, self.lens, self.slots
        width = len(old_pages[0])
        self.pages = [[old_pages[p][b] if p is not None and b * self.P < old_lens[p] and self.valid(old_pages[p][b]) else -1
                       for b in range(width)] for p in ok]
        self.lens = [old_lens[p] if p is not None else 0 for p in ok]
        for row in old_pages:
            for page in row:
                if self.valid(page):
                    self.refs[page] -= 1
        for row in self.pages:
            for page in row:
                if page >= 0:
                    self.refs[page] += 1
        left = iter([s for s in range(n) if s not in ok])
        taken, src, dst = set(), [-1] * n, [-1] * n
        self.slots = [0] * n
        for t, p in enumerate(ok):
            if p is not None and p not in taken:
                taken.add(p)
                self.slots[t] = old_slots[p]
                continue
            self.slots[t] = old_slots[next(left)]
            if p is not None and old_lens[p] > 0:
                src[t], dst[t] = old_slots[p], self.slots[t]
        return src, dst

    def reserve(self, new, max_len=1 << 30):
        """Lengths grow by `new`; copy_src, copy_dst, missing."""
        n = len(new)
        start = list(self.lens)
        self.lens = [a + b for a, b in zip(start, new)]
        wanted = []
        for s in range(n):
            end = min(self.lens[s], max_len, len(self.pages[s]) * self.P)
            if new[s] > 0 and end > start[s]:
                wanted += [(s, b) for b in range(start[s] // self.P, (end - 1) // self.P + 1)]
        held = list(self.refs)
        namers = {}
        for s, b in wanted:
            namers.setdefault(self.pages[s][b], []).append((s, b))
        free = iter([p for p in range(self.n_pages) if held[p] <= 0])
        src, dst, missing = [-1] * n, [-1] * n, [0] * n
        for s, b in wanted:
            page, partial = self.pages[s][b], b == start[s] // self.P and start[s] % self.P > 0
            if self.valid(page):
                if held[page] <= 1 or (len(namers[page]) == held[page] and namers[page][0] == (s, b)):
                    continue
            elif partial:
                missing[s] += 1
                continue
            got = next(free, -1)
            self.pages[s][b] = got
            if self.valid(page):
                self.refs[page] -= 1
            if got < 0:
                missing[s] += 1
                continue
            self.refs[got] = 1
            if self.valid(page) and partial and self.bits == 16:
                src[s], dst[s] = page, got
        return src, dst, missing

    def compact(self, max_moves):
        """copy_src, copy_dst, pages in use"""
        live = sum(r > 0 for r in self.refs)
        high = [p for p in range(self.n_pages - 1, live - 1, -1) if self.refs[p] > 0]
        low = [p for p in range(live) if self.refs[p] <= 0]
        moves = list(zip(high, low))[:max_moves]
        for a, b in moves:
            self.refs[b], self.refs[a] = self.refs[a], 0
        to = dict(moves)
        self.pages = [[to.get(p, p) for p in row] for row in self.pages]
        pad = [-1] * (max_moves - len(moves))
        return [a for a, _ in moves] + pad, [b for _, b in moves] + pad, live
