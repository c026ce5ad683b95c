"""Plain sequential definitions of the page operations (Python integers): the
map of a pool's pages, served row by row.  Shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np

PAGE = 16


def pages_for(n: int) -> int:
    return -(-n // PAGE)


class Map:
    """A page map; `bad` tells whether something was refused or out of range."""

    def __init__(self, table, blocks, refs):
        self.table, self.blocks, self.refs = (np.array(x, dtype=np.int64) for x in (table, blocks, refs))
        self.bad = False

    def held(self, p) -> bool:
        return 0 <= p < len(self.refs)

    def free(self, keep):
        for b, k in enumerate(keep):
            if k < 0:
                continue
            have = min(self.blocks[b], self.table.shape[1])
            for j in range(pages_for(int(k)), have):
                p = self.table[b, j]
                self.table[b, j] = -1
                if not self.held(p) or self.refs[p] <= 0:
                    self.bad = True
                else:
                    self.refs[p] -= 1
            if pages_for(int(k)) < have:
                self.blocks[b] = pages_for(int(k))

    def fork(self, lens, src, dst):
        """lens is changed in place."""
        rows = len(self.blocks)
        pairs = [(s, d) for s, d in zip(src, dst) if (s, d) != (-1, -1)]
        before = self.blocks.copy()
        for s, d in pairs:
            ok = 0 <= s < rows and 0 <= d < rows
            ok = ok and sum(e == d for _, e in pairs) == 1 and all(e != d for e, _ in pairs)
            n = pages_for(int(lens[s])) if ok else 0
            ok = ok and lens[s] >= 0 and n <= before[s] and n <= self.table.shape[1] and before[d] == 0
            if not ok or not all(self.held(p) and self.refs[p] > 0 for p in self.table[s, :n]):
                self.bad = True
                continue
            self.table[d, :n] = self.table[s, :n]
            self.refs[self.table[s, :n]] += 1
            self.blocks[d] = n
            lens[d] = lens[s]

    def reserve(self, lens, want):
        """(granted, copy_src, copy_dst), row by row; which rows are refused
        follows from the state that the call finds."""
        rows, width = self.table.shape
        nobody = {p for p in range(len(self.refs)) if self.refs[p] <= 0}
        granted, src, dst = [0] * rows, [-1] * rows, [-1] * rows
        stopped = False
        for b in range(rows):
            n, w, have = int(lens[b]), int(want[b]), int(self.blocks[b])
            if w <= n:
                granted[b] = 1
                continue
            need = pages_for(w)
            if n < 0 or have < 0 or have > width or need > width or pages_for(n) > have:
                self.bad = True
                continue
            span = range(n // PAGE, min(have, need))
            if not all(self.held(self.table[b, j]) and self.table[b, j] not in nobody for j in span):
                self.bad = True
                continue
            if stopped:
                continue
            anew = [j for j in span if self.refs[self.table[b, j]] > 1]
            places = anew + list(range(have, need))
            free = [p for p in range(len(self.refs)) if self.refs[p] == 0][:len(places)]
            if len(free) < len(places):
                stopped = True
                continue
            for j, p in zip(places, free):
                if j < have:
                    old = self.table[b, j]
                    self.refs[old] -= 1
                    if j == n // PAGE and n % PAGE:
                        src[b], dst[b] = int(old), p
                self.table[b, j] = p
                self.refs[p] = 1
            self.blocks[b] = max(have, need)
            granted[b] = 1
        return granted, src, dst

    def compact(self):
        """(moves as (source, target) pairs, remap)."""
        live = [p for p in range(len(self.refs)) if self.refs[p] > 0]
        n = len(live)
        moves = list(zip([p for p in live if p >= n], [p for p in range(n) if self.refs[p] <= 0]))
        remap = [-1] * len(self.refs)
        for p in live:
            remap[p] = p
        for s, d in moves:
            remap[s] = d
            self.refs[d], self.refs[s] = self.refs[s], 0
        for b in range(len(self.blocks)):
            for j in range(min(self.blocks[b], self.table.shape[1])):
                p = self.table[b, j]
                if self.held(p) and remap[p] >= 0:
                    self.table[b, j] = remap[p]
                else:
                    self.bad = True
        return moves, remap
