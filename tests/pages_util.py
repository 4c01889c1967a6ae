"""A page pool kept one page at a time: what the GPU's books and pages are held to."""
import numpy as np


class Books:
    def __init__(self, refs, lens, tables, pages, page_tokens):
        self.refs, self.lens, self.tables, self.pages, self.pt = refs, lens, tables, pages, page_tokens

    def slots(self, n):
        return -(-int(n) // self.pt)

    def fork(self, rows, parents, lens):
        """False where the request is refused (nothing changed)."""
        B, T = self.tables.shape
        old_lens, old_tables = self.lens.copy(), self.tables.copy()
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        plan, seen = [], set()
        for row, par, n in zip(rows, parents, lens):
            if not (0 <= row < B and -1 <= par < B and 0 <= n <= T * self.pt) or row in seen:
                return False
            seen.add(row)
            have = 0 if par < 0 else int(old_lens[par])
            if (n < have) if par == row else old_lens[row] != 0:
                return False
            first = self.slots(have) if par == row else min(have, n) // self.pt
            part = par != row and min(have, n) % self.pt != 0
            plan.append((row, par, n, first, part))
        if sum(self.slots(n) - first for _, _, n, first, _ in plan) > len(free):
            return False
        for row, par, n, first, part in plan:
            if par != row:
                for s in range(first):
                    self.tables[row, s] = old_tables[par, s]
                    self.refs[old_tables[par, s]] += 1
            for s in range(first, self.slots(n)):
                p = free.pop(0)
                self.tables[row, s], self.refs[p] = p, 1
                if s == first and part:
                    self.pages[:, p] = self.pages[:, old_tables[par, s]]
            self.lens[row] = n
        return True

    def free(self, rows):
        for row in rows:
            for s in range(self.slots(self.lens[row])):
                self.refs[self.tables[row, s]] -= 1
                self.tables[row, s] = -1
            self.lens[row] = 0

    def compact(self):
        live = int((self.refs > 0).sum())
        holes = [p for p in range(live) if self.refs[p] == 0]
        to = np.arange(len(self.refs), dtype=np.int32)
        for p in range(live, len(self.refs)):
            if self.refs[p] > 0:
                h = holes.pop(0)
                self.pages[:, h] = self.pages[:, p]
                self.refs[h], self.refs[p] = self.refs[p], 0
                to[p] = h
        self.tables[:] = np.where(self.tables >= 0, to[self.tables], -1)
        return live


def empty(pages, page_tokens, seqs, slots):
    return Books(np.zeros(pages.shape[1], np.int32), np.zeros(seqs, np.int32), np.full((seqs, slots), -1, np.int32), pages, page_tokens)
