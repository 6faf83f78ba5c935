"""Plain Python model of the page calls (include/tq.h): lists and loops."""
import numpy as np


class Pool:
    def __init__(self, n_pages, page_tokens, n_seqs, cols):
        self.pt, self.cols = page_tokens, cols
        self.table = np.full((n_seqs, cols), -1, np.int32)
        self.lens = np.zeros(n_seqs, np.int32)
        self.refs = np.zeros(n_pages, np.int32)

    def copy(self):
        c = Pool(len(self.refs), self.pt, len(self.lens), self.cols)
        c.table, c.lens, c.refs = self.table.copy(), self.lens.copy(), self.refs.copy()
        return c

    def held(self, n):
        return -(-int(n) // self.pt)

    def free_pages(self):
        return [int(p) for p in np.nonzero(self.refs == 0)[0]]

    def extend(self, seqs, n_new):
        """True when no entry was skipped."""
        ok, free, at, seen = True, self.free_pages(), 0, set()
        for s, add in zip(seqs, n_new):
            if not 0 <= s < len(self.lens) or s in seen or add < 0 or self.lens[s] + add > self.cols * self.pt:
                ok = False
                if 0 <= s < len(self.lens):
                    seen.add(s)
                continue
            seen.add(s)
            p0, p1 = self.held(self.lens[s]), self.held(self.lens[s] + add)
            first, at = at, at + p1 - p0
            if p1 > p0 and at > len(free):
                ok = False
                continue
            for j in range(p0, p1):
                self.table[s, j] = free[first + j - p0]
                self.refs[free[first + j - p0]] = 1
            self.lens[s] += add
        return ok

    def free(self, seqs):
        ok = True
        for s in seqs:
            if not 0 <= s < len(self.lens):
                ok = False
                continue
            for j in range(self.held(self.lens[s])):
                self.refs[self.table[s, j]] -= 1
                self.table[s, j] = -1
            self.lens[s] = 0
        return ok

    def fork(self, pools, parents, children):
        """pools: uint8 arrays [n_pages, page_tokens, row_bytes]."""
        ok, free, at, seen = True, self.free_pages(), 0, set()
        lens = self.lens.copy()
        for p, c in zip(parents, children):
            bad = not 0 <= p < len(lens) or not 0 <= c < len(lens) or lens[c] != 0 or c in seen
            if 0 <= c < len(lens):
                seen.add(c)
            if bad:
                ok = False
                continue
            n = int(lens[p])
            whole, rest = divmod(n, self.pt)
            if rest:
                at += 1
                if at > len(free):
                    ok = False
                    continue
            self.table[c, :whole] = self.table[p, :whole]
            for q in self.table[p, :whole]:
                self.refs[q] += 1
            if rest:
                page = free[at - 1]
                self.table[c, whole], self.refs[page] = page, 1
                for x in pools:
                    x[page, :rest] = x[self.table[p, whole], :rest]
            self.lens[c] = n
        return ok

    def compact(self, pools):
        used = np.nonzero(self.refs > 0)[0]
        U = len(used)
        holes = [p for p in range(U) if self.refs[p] == 0]
        movers = [int(p) for p in used if p >= U]
        new = np.arange(len(self.refs))
        new[movers] = holes
        for h, m in zip(holes, movers):
            for x in pools:
                x[h] = x[m]
            self.refs[h], self.refs[m] = self.refs[m], 0
        self.table = np.where(self.table >= 0, new[np.maximum(self.table, 0)], -1).astype(np.int32)
        return U
