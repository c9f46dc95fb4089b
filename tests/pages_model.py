"""The calls on a cache's pages as plain Python on lists: what the kernels are held against."""


class Model:
    def __init__(self, seqs, ldt, pages, ps):
        self.len = [0] * seqs
        self.table = [[-1] * ldt for _ in range(seqs)]
        self.refs = [0] * pages
        self.seqs, self.ldt, self.pages, self.ps = seqs, ldt, pages, ps

    def _length(self, s):
        return max(0, min(self.len[s], self.ldt * self.ps))

    def _held(self, tokens):
        return -(-tokens // self.ps)

    def _free(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def grow(self, seq, add):
        free, taken, seen, got = self._free(), 0, set(), []
        for s, a in zip(seq, add):
            first = s not in seen
            seen.add(s)
            if not 0 <= s < self.seqs:
                got.append(0)
                continue
            old = self._length(s)
            self.len[s] = old
            if not first or a <= 0 or old + a > self.ldt * self.ps:
                got.append(0)
                continue
            need = self._held(old + a) - self._held(old)
            taken += need
            if need and taken > len(free):
                got.append(0)
                continue
            for j, p in enumerate(free[taken - need:taken]):
                self.table[s][self._held(old) + j] = p
                self.refs[p] = 1
            self.len[s] = old + a
            got.append(a)
        return got

    def fork(self, parent, child):
        free, taken, seen, src, dst = self._free(), 0, set(), [], []
        before = [self._length(s) for s in range(self.seqs)]
        for p, c in zip(parent, child):
            ok = 0 <= p < self.seqs and 0 <= c < self.seqs and before[c] == 0
            if ok:
                self.len[c] = 0 if c not in seen else self.len[c]
                ok = c not in seen
                seen.add(c)
            n = before[p] if ok else 0
            cut = ok and n % self.ps != 0
            if cut:
                taken += 1
                ok = taken <= len(free)
            if not ok:
                src.append(-2)
                dst.append(-2)
                continue
            self.len[c] = n
            for j in range(n // self.ps):
                self.table[c][j] = self.table[p][j]
                self.refs[self.table[p][j]] += 1
            if cut:
                page = free[taken - 1]
                self.table[c][n // self.ps] = page
                self.refs[page] = 1
            src.append(self.table[p][n // self.ps] if cut else -1)
            dst.append(page if cut else -1)
        return src, dst

    def free(self, seq):
        for s in seq:
            if 0 <= s < self.seqs:
                for j in range(self._held(self._length(s))):
                    if 0 <= self.table[s][j] < self.pages:
                        self.refs[self.table[s][j]] -= 1
                    self.table[s][j] = -1
                self.len[s] = 0

    def compact(self):
        """(table, refs, src, dst, live) after the move."""
        live = sum(r != 0 for r in self.refs)
        hole = [p for p in range(live) if self.refs[p] == 0]
        mover = [p for p in range(live, self.pages) if self.refs[p] != 0]
        to = {p: p for p in range(live) if self.refs[p] != 0}
        to.update(zip(mover, hole))
        refs = [0] * self.pages
        for p, q in to.items():
            refs[q] = self.refs[p]
        pad = [-1] * (self.pages // 2 - len(mover))
        return [[to.get(p, -1) for p in r] for r in self.table], refs, mover + pad, hole + pad, live

    def slots(self, start, kvheads):
        """Cache rows of each row's token and head; None where a row belongs to no sequence."""
        rows = start[-1] if start else self.seqs
        out = [None] * (rows * kvheads)
        for s in range(self.seqs):
            a, b = (start[s], start[s + 1]) if start else (s, s + 1)
            for r in range(a, b):
                t = self._length(s) - (b - r)
                page = self.table[s][t // self.ps] if t >= 0 else -1
                for h in range(kvheads):
                    ok = 0 <= page < self.pages
                    out[r * kvheads + h] = (page * kvheads + h) * self.ps + t % self.ps if ok else -1
        return out
