"""The state of a paged cache as Python lists, and its operations from their definitions."""


class Pool:
    def __init__(self, batch, most, n_pages, block):
        self.batch, self.most, self.block = batch, most, block
        self.table = [[-1] * most for _ in range(batch)]
        self.seqlens = [0] * batch
        self.refs = [0] * n_pages

    def blocks(self, b):
        return -(-self.seqlens[b] // self.block)

    def fork(self, src, dst):
        old = [(list(self.table[s]), self.seqlens[s], self.blocks(s)) for s in src]
        for (row, n, nb), s, d in zip(old, src, dst):
            if s == d:
                continue
            for p in row[:nb]:
                self.refs[p] += 1
            self._set(d, row[:nb], n)

    def _set(self, d, pages, n):
        had = self.blocks(d)
        for p in self.table[d][:had]:
            self.refs[p] -= 1
        for c in range(max(had, len(pages))):
            self.table[d][c] = pages[c] if c < len(pages) else -1
        self.seqlens[d] = n

    def free(self, slots):
        for d in slots:
            self._set(d, [], 0)

    def grow(self, n_new):
        """-> copy_src, copy_dst, or None when the pool has too few free pages."""
        free = [p for p, r in enumerate(self.refs) if r == 0]
        refs, rows = list(self.refs), [list(r) for r in self.table]
        src, dst = [-1] * self.batch, [-1] * self.batch
        for b, n in enumerate(n_new):
            if n == 0:
                continue
            nb, after = self.blocks(b), -(-(self.seqlens[b] + n) // self.block)
            want = after - nb
            last = rows[b][nb - 1] if nb else -1
            copy = self.seqlens[b] % self.block != 0 and refs[last] > 1
            if want + copy > len(free):
                return None
            if copy:
                page = free.pop(0)
                refs[last] -= 1
                refs[page] = 1
                rows[b][nb - 1] = page
                src[b], dst[b] = last, page
            for c in range(nb, after):
                rows[b][c] = free.pop(0)
                refs[rows[b][c]] = 1
        self.refs, self.table = refs, rows
        self.seqlens = [s + n for s, n in zip(self.seqlens, n_new)]
        return src, dst

    def compact(self):
        """-> moves (src, dst), pages in use."""
        held = sum(r > 0 for r in self.refs)
        src = [p for p in range(held, len(self.refs)) if self.refs[p] > 0]
        dst = [p for p in range(held) if self.refs[p] == 0]
        to = dict(zip(src, dst))
        for s, d in zip(src, dst):
            self.refs[d], self.refs[s] = self.refs[s], 0
        for b in range(self.batch):
            for c in range(self.blocks(b)):
                self.table[b][c] = to.get(self.table[b][c], self.table[b][c])
        return src, dst, held

    def counted(self):
        """How often each page is held, counted from the table."""
        n = [0] * len(self.refs)
        for b in range(self.batch):
            for p in self.table[b][:self.blocks(b)]:
                n[p] += 1
        return n
