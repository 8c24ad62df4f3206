"""A plain model of pages that requests share, for the tests: lists and counts."""
from __future__ import annotations


def up(n, ps):
    return -(-n // ps)


class Pool:
    """Tables, counts and free stack; step() and compact() return the pages to copy, or None where the step does not fit."""

    def __init__(self, n_req, n_pages, max_pages, ps, free=None, refs=None):
        self.ps, self.n_pages, self.max_pages = ps, n_pages, max_pages
        self.table = [[0] * max_pages for _ in range(n_req)]
        self.held = [0] * n_req  # tokens
        self.free = list(range(n_pages)) if free is None else list(free)
        self.refs = [0] * n_pages if refs is None else list(refs)

    def step(self, q, kv, src):
        ps, n = self.ps, len(q)
        old = [row[:] for row in self.table]
        keep = [min(up(self.held[s], ps), up(max(0, kv[r] - q[r]), ps)) if s >= 0 else 0 for r, s in enumerate(src)]
        total, seen = self.refs[:], {}
        for r in range(n):
            for page in old[r][:up(self.held[r], ps)]:
                total[page] -= 1
                seen.setdefault(page)
        rows = [old[src[r]][:keep[r]] if src[r] >= 0 else [] for r in range(n)]
        for row in rows:
            for page in row:
                total[page] += 1
        stack = self.free + [page for page in seen if total[page] == 0]
        writers = {}
        at = [None] * n
        for r in range(n):
            w = max(0, kv[r] - q[r])
            if q[r] > 0 and w < kv[r] and w % ps and w // ps < keep[r]:
                at[r] = w // ps
                writers.setdefault(rows[r][at[r]], []).append(r)
        refs, copies = total[:], []
        for r in range(n):
            if at[r] is not None:
                page = rows[r][at[r]]
                if not (len(writers[page]) == total[page] and writers[page][0] == r):
                    if not stack:
                        return None
                    rows[r][at[r]] = stack.pop()
                    copies.append([page, rows[r][at[r]]])
                    refs[page] -= 1
                    refs[rows[r][at[r]]] += 1
            for _ in range(keep[r], up(kv[r], ps)):
                if not stack:
                    return None
                rows[r].append(stack.pop())
                refs[rows[r][-1]] += 1
        for r in range(n):
            self.table[r][:len(rows[r])] = rows[r]
            if len(rows[r]) > up(kv[r], ps):  # cannot be: keep <= need
                raise AssertionError
        self.refs, self.free, self.held = refs, stack, list(kv)
        return copies

    def slots(self, q, kv, T):
        out = []
        for r in range(len(q)):
            for i in range(q[r]):
                pos = kv[r] - q[r] + i
                out.append(self.table[r][pos // self.ps] * self.ps + pos % self.ps if pos >= 0 else -1)
        return out + [-1] * (T - len(out))

    def compact(self):
        used = self.n_pages - len(self.free)
        free = set(self.free)
        moves = list(zip([i for i in range(used, self.n_pages) if i not in free], [i for i in range(used) if i in free]))
        to = dict(moves)
        for r, row in enumerate(self.table):
            for k in range(up(self.held[r], self.ps)):
                row[k] = to.get(row[k], row[k])
        for a, b in moves:
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.free = [self.n_pages - 1 - i for i in range(len(self.free))]
        return [list(m) for m in moves]
