"""The bookkeeping of a paged key/value cache, followed entry by entry on the host (test
infrastructure only): what attn_kv_reserve, attn_kv_fork, attn_kv_free, attn_kv_evict and
attn_kv_compact make of a page table, lengths and counts."""
from __future__ import annotations

import copy


class Pages:
    def __init__(self, S, max_pages, n_pages, page):
        self.table = [[-1] * max_pages for _ in range(S)]
        self.lens = [0] * S
        self.refs = [0] * n_pages
        self.page = page

    def copy(self):
        return copy.deepcopy(self)

    def _free(self):
        return [x for x, r in enumerate(self.refs) if r == 0]

    def reserve(self, n_new):
        """The first new token's position for every sequence, or None when refused."""
        page, M = self.page, len(self.table[0])
        need = []
        for s, n in enumerate(n_new):
            if n < 0 or self.lens[s] + n > M * page:
                return None
            need.append(-(-(self.lens[s] + n) // page) + -self.lens[s] // page)
        free = self._free()
        if sum(need) > len(free):
            return None
        start = self.lens[:len(n_new)]
        for s, n in enumerate(n_new):
            for i in range(need[s]):
                x = free.pop(0)
                self.table[s][-(-start[s] // page) + i] = x
                self.refs[x] = 1
            self.lens[s] += n
        return start

    def fork(self, parents, children):
        """(copy_src, copy_dst), or None when refused."""
        S = len(self.lens)
        if len(set(children)) != len(children) or set(parents) & set(children):
            return None
        if any(not 0 <= x < S for x in parents + children) or any(self.lens[c] for c in children):
            return None
        part = [self.lens[a] % self.page > 0 for a in parents]
        free = self._free()
        if sum(part) > len(free):
            return None
        src, dst = [], []
        for a, c, own in zip(parents, children, part):
            full = self.lens[a] // self.page
            row = [-1] * len(self.table[c])
            for m in range(full):
                row[m] = self.table[a][m]
                if row[m] >= 0:
                    self.refs[row[m]] += 1
            src.append(self.table[a][full] if own else -1)
            dst.append(free.pop(0) if own else -1)
            if own:
                row[full] = dst[-1]
                self.refs[dst[-1]] = 1
            self.table[c] = row
            self.lens[c] = self.lens[a]
        return src, dst

    def free(self, seqs):
        for s in set(seqs):
            for m, x in enumerate(self.table[s]):
                if x >= 0:
                    self.refs[x] -= 1
                self.table[s][m] = -1
            self.lens[s] = 0

    def evict(self, window, sinks):
        for s, row in enumerate(self.table):
            for m, x in enumerate(row):
                keys = range(m * self.page, (m + 1) * self.page)
                if x >= 0 and keys[0] >= sinks and keys[-1] < self.lens[s] - window:
                    self.refs[x] -= 1
                    row[m] = -1

    def compact(self):
        """(copy_src, copy_dst), without the tail of -1."""
        live = sum(r > 0 for r in self.refs)
        dst = [x for x in range(live) if self.refs[x] == 0]
        src = [x for x in range(live, len(self.refs)) if self.refs[x] > 0]
        to = dict(zip(src, dst))
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.table = [[to.get(x, x) for x in row] for row in self.table]
        return src, dst
