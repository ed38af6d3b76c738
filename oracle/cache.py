"""Plain CPU oracle of the paged cache and of the attention over it (numpy, float64).

TEST INFRASTRUCTURE ONLY (see the package docstring).

``Book`` keeps a cache's bookkeeping one request after the other, as a host would; ``attention``
computes the new tokens' outputs from gathered rows.
"""
from __future__ import annotations

import numpy as np

PAGE, CAPACITY, LENGTH, FORK, LAYOUT, TREE = 32, 64, 128, 256, 1, 16


def pages_of(tokens, page_size):
    return -(-int(tokens) // page_size)


class Book:
    """Tables, lengths and counts of a cache, with the rows it copies or moves listed."""

    def __init__(self, requests, max_pages, num_pages, page_size):
        self.P, self.MP = page_size, max_pages
        self.table = np.full((requests, max_pages), -1, np.int32)
        self.lens = np.zeros(requests, np.int32)
        self.held = np.zeros(requests, np.int32)
        self.ref = np.zeros(num_pages, np.int32)
        self.free = np.arange(num_pages, dtype=np.int32)
        self.num_free = num_pages
        self.bits, self.first = 0, 2 ** 31 - 1

    def _error(self, bits, request=None):
        self.bits |= bits
        if request is not None:
            self.first = min(self.first, int(request))

    def take_error(self):
        got = (self.bits, -1 if self.first == 2 ** 31 - 1 else self.first)
        self.bits, self.first = 0, 2 ** 31 - 1
        return got

    def slot(self, r, pos):
        return int(self.table[r, pos // self.P]), int(pos % self.P)

    def reserve(self, n):
        """Returns the row copies [(old page, new page, rows)]."""
        plan, need_free, first_short = [], 0, None
        left = {}
        for r, m in enumerate(n):
            if m <= 0:
                continue
            length = int(self.lens[r])
            if length < 0 or length > self.held[r] * self.P or length + m > self.MP * self.P:
                self._error(LENGTH, r)
                continue
            copy = None
            if length % self.P:
                page = int(self.table[r, length // self.P])
                if not 0 <= page < len(self.ref) or self.ref[page] < 1:
                    self._error(PAGE, r)
                    continue
                others = left.get(page, int(self.ref[page]))
                if others > 1:
                    copy = page
                    left[page] = others - 1
            fresh = max(pages_of(length + m, self.P) - int(self.held[r]), 0) + (copy is not None)
            need_free += fresh
            if first_short is None and fresh and need_free > self.num_free:
                first_short = r
            plan.append((r, m, copy))
        if need_free > self.num_free:
            self._error(CAPACITY, first_short)
            return []
        copies = []

        def pop():
            self.num_free -= 1
            page = int(self.free[self.num_free])
            self.ref[page] = 1
            return page

        for r, m, copy in plan:
            length = int(self.lens[r])
            if copy is not None:
                new = pop()
                self.ref[copy] -= 1
                self.table[r, length // self.P] = new
                copies.append((copy, new, length % self.P))
            while self.held[r] < pages_of(length + m, self.P):
                self.table[r, self.held[r]] = pop()
                self.held[r] += 1
        return copies

    def commit(self, n, accepted, parents=None, last=None):
        """Returns the row moves [(request, from position, to position)]; ``parents`` per request."""
        moves = []
        for r, m in enumerate(n):
            a = int(accepted[r])
            if m == 0 or a == -1:
                continue
            length = int(self.lens[r])
            held = int(self.held[r])
            if a < -1 or a >= m or length < 0 or not 0 <= held <= self.MP or length + m > held * self.P:
                self._error(LENGTH, r)
                continue
            if parents is not None:
                path, at, par = [], int(last[r]), parents[r]
                while 0 <= at < m and len(path) <= a:
                    path.append(at)
                    if not (par[at] == -1 if at == 0 else 0 <= par[at] < at):
                        break
                    at = int(par[at])
                if m > 128 or len(path) != a + 1 or path[-1] != 0:
                    self._error(TREE, r)
                    continue
                moves += [(r, length + node, length + d) for d, node in enumerate(reversed(path)) if node != d]
            self.lens[r] = length + a + 1
        return moves

    def fork(self, src, dst):
        bad = [not (0 <= s < len(self.lens) and 0 <= d < len(self.lens)) or list(dst).count(d) > 1 or
               s in dst or d in src or self.held[d] != 0 for s, d in zip(src, dst)]
        for s, d, b in zip(src, dst, bad):
            if b:
                self._error(FORK, d if 0 <= d < len(self.lens) else None)
                continue
            count = pages_of(self.lens[s], self.P) if self.lens[s] >= 0 else -1
            if count < 0 or count > self.held[s]:
                self._error(LENGTH, d)
                continue
            pages = self.table[s, :count]
            if ((pages < 0) | (pages >= len(self.ref))).any() or (self.ref[pages] < 1).any():
                self._error(PAGE, d)
                continue
            self.table[d, :count] = pages
            self.ref[pages] += 1
            self.lens[d], self.held[d] = self.lens[s], count

    def release(self, keep=None, B=None):
        freed = []
        for r in range(len(self.lens) if B is None else B):
            want = int(self.lens[r] if keep is None else keep[r])
            if want < 0 or self.lens[r] < 0 or not 0 <= self.held[r] <= self.MP:
                self._error(LENGTH, r)
                continue
            self.lens[r] = min(int(self.lens[r]), want)
            kept = pages_of(self.lens[r], self.P)
            for i in range(kept, int(self.held[r])):
                page = int(self.table[r, i])
                self.table[r, i] = -1
                if not 0 <= page < len(self.ref) or self.ref[page] < 1:
                    self._error(PAGE, r)
                    continue
                self.ref[page] -= 1
                if self.ref[page] == 0:
                    freed.append(page)
            self.held[r] = min(int(self.held[r]), kept)
        for page in sorted(freed):
            self.free[self.num_free] = page
            self.num_free += 1


def visible(n, ctx, parent=None):
    """[n, ctx + n] which positions each new token sees."""
    seen = np.ones((n, ctx + n), bool)
    seen[:, ctx:] = np.tril(np.ones((n, n), bool)) if parent is None else False
    if parent is not None:
        for i in range(n):
            if parent[i] >= 0:
                seen[i, ctx:] = seen[parent[i], ctx:]
            seen[i, ctx + i] = True
    return seen


def attention(q, k, v, seen, scale):
    """One request, one kv head: q [n, G, D], k and v [L, D], seen [n, L].  Returns out [n, G, D],
    lse [n, G], and per output the sums that bound the error of a computation in fewer bits:
    mass = sum p |v| [n, G, D] and reach = max over visible keys of scale * sum |q| |k| [n, G]."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    s = np.einsum("igd,td->igt", q, k) * scale
    s = np.where(seen[:, None, :], s, -np.inf)
    top = s.max(-1, keepdims=True)
    p = np.exp(s - top)
    total = p.sum(-1, keepdims=True)
    p /= total
    reach = np.where(seen[:, None, :], np.einsum("igd,td->igt", np.abs(q), np.abs(k)) * scale, 0).max(-1)
    return (np.einsum("igt,td->igd", p, v), (top + np.log(total))[..., 0],
            np.einsum("igt,td->igd", p, np.abs(v)), reach)
