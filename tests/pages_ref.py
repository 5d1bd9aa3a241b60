"""The page pool from its definition: lists of page ids, one slot and one page at a time."""
from __future__ import annotations


class Pool:
    def __init__(self, rows, lens, ref, page, width):
        self.rows = [list(r) for r in rows]  # pages of each slot's tokens
        self.lens, self.ref, self.page, self.width = list(lens), list(ref), page, width

    def table(self):
        return [r + [-1] * (self.width - len(r)) for r in self.rows]

    def pages(self, tokens):
        return -(-tokens // self.page)

    def fork(self, parent, added, keep=None):
        """(status bits, moves, cu_q); nothing changes where a bit is set."""
        n = len(self.rows)
        none = [(-1, -1, -1)] * n, [0] * (n + 1)
        if any(not -1 <= p < n for p in parent) or any(a < 0 for a in added):
            return 2, *none
        kept = [0 if p < 0 else self.lens[p] if keep is None else min(max(keep[i], 0), self.lens[p])
                for i, p in enumerate(parent)]
        if any(k + a > self.width * self.page for k, a in zip(kept, added)):
            return 2, *none
        rows = [self.rows[p][:self.pages(k)] if p >= 0 else [] for p, k in zip(parent, kept)]
        ref = list(self.ref)
        for r in self.rows:
            for x in r:
                ref[x] -= 1
        for r in rows:
            for x in r:
                ref[x] += 1
        writes = [k % self.page != 0 and a > 0 for k, a in zip(kept, added)]
        writers = {}
        for i in range(n):
            if writes[i]:
                writers.setdefault(rows[i][-1], []).append(i)
        free, moves, uses = [x for x in range(len(ref)) if ref[x] == 0], [], list(ref)
        for i in range(n):
            if writes[i]:
                x = rows[i][-1]
                if ref[x] > 1 and not (len(writers[x]) == ref[x] and writers[x][0] == i):
                    if not free:
                        return 8, *none
                    rows[i][-1] = free.pop(0)
                    uses[x] -= 1
                    uses[rows[i][-1]] = 1
                    moves.append((x, rows[i][-1], kept[i] % self.page))
            while len(rows[i]) < self.pages(kept[i] + added[i]):
                if not free:
                    return 8, *none
                rows[i].append(free.pop(0))
                uses[rows[i][-1]] = 1
        self.rows, self.ref, self.lens = rows, uses, [k + a for k, a in zip(kept, added)]
        cu = [0]
        for a in added:
            cu.append(cu[-1] + a)
        return 0, moves + [(-1, -1, -1)] * (n - len(moves)), cu

    def compact(self):
        used = [x for x, u in enumerate(self.ref) if u != 0]
        holes = [x for x, u in enumerate(self.ref) if u == 0 and x < len(used)]
        to = dict(zip(used[len(used) - len(holes):], holes))
        for src, dst in to.items():
            self.ref[dst], self.ref[src] = self.ref[src], 0
        self.rows = [[to.get(x, x) for x in r] for r in self.rows]
        moves = [(src, dst, self.page) for src, dst in to.items()]
        return moves + [(-1, -1, -1)] * (len(self.ref) // 2 - len(moves))
