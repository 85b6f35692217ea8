"""Plain forms of the pages' bookkeeping (Python), for its tests: the pool, the
block table and the lengths as lists, one sequence after the other."""


class Pool:
    def __init__(self, pages, B, columns, page):
        self.refs, self.page, self.columns = [0] * pages, page, columns
        self.table = [[0] * columns for _ in range(B)]
        self.len = [0] * B

    def pages(self, n):
        return -(-n // self.page)

    def fork(self, parents, children):
        for p, c in zip(parents, children):
            n = self.pages(self.len[p])
            self.table[c][:n] = self.table[p][:n]
            for x in self.table[p][:n]:
                self.refs[x] += 1
            self.len[c] = self.len[p]

    def release(self, ids, keep=None):
        for i, b in enumerate(ids):
            to = keep[i] if keep else 0
            for x in self.table[b][self.pages(to):self.pages(self.len[b])]:
                self.refs[x] -= 1
            self.len[b] = to

    def reserve(self, new):
        """(slots, copies), or None where there is no room (nothing changes)."""
        free = [p for p, r in enumerate(self.refs) if r == 0]
        refs, table = list(self.refs), [list(r) for r in self.table]
        slots, copies, at = [], [], 0

        def take():
            nonlocal at
            at += 1
            return free[at - 1] if at <= len(free) else None
        for b, n in enumerate(new):
            pair = (-1, -1)
            if n and self.pages(self.len[b] + n) > self.columns:
                return None
            for i in range(self.len[b], self.len[b] + n):
                c = i // self.page
                if i % self.page == 0 or refs[table[b][c]] > 1 and i == self.len[b]:
                    p = take()
                    if p is None:
                        return None
                    if i % self.page:
                        pair = (table[b][c], p)
                        refs[pair[0]] -= 1
                    refs[p] = 1
                    table[b][c] = p
                slots.append(table[b][c] * self.page + i % self.page)
            copies.append(pair)
        self.refs, self.table = refs, table
        self.len = [a + n for a, n in zip(self.len, new)]
        return slots, copies
