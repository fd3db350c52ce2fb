"""CPU oracle of the paged-cache operators: plain, slow, fp64 and Python integers.

TEST INFRASTRUCTURE, as ``bsa_oracle``: only the tests and the package smoke check import it,
and it imports nothing from the product. Pools are numpy fp64 arrays (the 16-bit values widened exactly): K, V
[n_pages, Hkv, page, d], bounds [n_pages, Hkv, 2, d]; tables are lists of lists of page numbers.
"""
from __future__ import annotations

import numpy as np


class Book:
    """Page table, lengths and reference counts."""

    def __init__(self, slots, max_pages, n_pages, page):
        self.page, self.max_pages, self.n_pages = page, max_pages, n_pages
        self.table = [[-1] * max_pages for _ in range(slots)]
        self.len = [0] * slots
        self.refs = [0] * n_pages

    def pages(self, n):
        return -(-n // self.page)

    def fork(self, parent):
        """Returns True when every fork was allowed."""
        ok = True
        before = list(self.len)
        for c, p in enumerate(parent):
            if p < 0:
                continue
            if p >= len(self.table) or p == c or parent[p] >= 0 or before[c] != 0:
                ok = False
                continue
            n = self.pages(self.len[p])
            self.table[c] = self.table[p][:n] + [-1] * (self.max_pages - n)
            for pg in self.table[c][:n]:
                self.refs[pg] += 1
            self.len[c] = self.len[p]
        return ok

    def resize(self, new_len):
        """Returns (pairs, free pages, pages ran out, bad length)."""
        S = len(self.table)
        bad = any(n > self.max_pages * self.page for n in new_len)
        want = [(-1 if n > self.max_pages * self.page else n) for n in new_len]
        for s, n in enumerate(want):
            if 0 <= n < self.len[s]:
                for j in range(self.pages(n), self.pages(self.len[s])):
                    self.refs[self.table[s][j]] -= 1
                    self.table[s][j] = -1
                self.len[s] = n
        grow = [s for s in range(S) if want[s] > self.len[s]]
        tail = {}
        for s in grow:
            if self.len[s] % self.page:
                pg = self.table[s][self.len[s] // self.page]
                if self.refs[pg] > 1:
                    tail[s] = pg
        keeper = set()
        for s, pg in tail.items():
            same = [u for u in tail if tail[u] == pg]
            if len(same) == self.refs[pg] and s == max(same):
                keeper.add(s)
        free = [p for p in range(self.n_pages) if self.refs[p] == 0]
        pairs = [(-1, -1)] * S
        short, used, out = False, 0, 0
        for s in grow:
            copy = s in tail and s not in keeper
            need = self.pages(want[s]) - self.pages(self.len[s]) + copy
            out += need
            if (need or s in keeper) and out > len(free):
                short = True
                continue
            mine = free[out - need:out]
            used += need
            for pg in mine:
                self.refs[pg] = 1
            if copy:
                old = tail[s]
                self.refs[old] -= 1
                pairs[s] = (old, mine[0])
                self.table[s][self.len[s] // self.page] = mine[0]
                mine = mine[1:]
            for i, pg in enumerate(mine):
                self.table[s][self.pages(self.len[s]) + i] = pg
            self.len[s] = want[s]
        return pairs, len(free) - used, short, bad


def rows_of(pool, table, n, page, h):
    """The first n rows of a sequence, head h."""
    return np.stack([pool[table[p // page], h, p % page] for p in range(n)]) if n else \
        np.zeros((0, pool.shape[-1]))


def ancestors(parents):
    """bool [T, T]: token t sees j (itself and its ancestors)."""
    T = len(parents)
    see = np.zeros((T, T), bool)
    for t in range(T):
        x = t
        while x >= 0:
            see[t, x] = True
            x = parents[x]
    return see


def softmax_rows(q, k, v, see, scale):
    """q [R, d], k, v [n, d], see [R, n]: (output, lse); only the pairs seen take part."""
    out = np.zeros((q.shape[0], v.shape[1]))
    lse = np.full(q.shape[0], -np.inf)
    for r in range(q.shape[0]):
        at = np.nonzero(see[r])[0]
        if len(at) == 0:
            continue
        z = scale * (k[at] @ q[r])
        m = z.max()
        p = np.exp(z - m)
        out[r] = p @ v[at] / p.sum()
        lse[r] = m + np.log(p.sum())
    return out, lse


def attend_tree(q, k, v, table, n, ql, page, see_drafts, scale):
    """One slot: q [Hq, ql, d] -> (out [Hq, ql, d], lse [Hq, ql]). see_drafts bool [ql, ql]."""
    Hq, Hkv = q.shape[0], k.shape[1]
    out, lse = np.zeros(q.shape), np.zeros(q.shape[:2])
    see = np.concatenate([np.ones((ql, n - ql), bool), see_drafts], 1)
    for h in range(Hkv):
        kr, vr = rows_of(k, table, n, page, h), rows_of(v, table, n, page, h)
        for g in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
            out[g], lse[g] = softmax_rows(q[g], kr, vr, see, scale)
    return out, lse


def page_score(qg, lo, hi):
    """qg [G, d], lo, hi [d]: the fp32 score of a page for the heads of a group."""
    return np.float32(max(np.maximum(x * lo, x * hi).sum() for x in qg))


def select(scores, own_page, k, n_first, n_last):
    """scores: fp32 of pages 0 .. own_page. The ascending list of selected pages."""
    vis = own_page + 1
    must = [j for j in range(vis) if j < n_first or j >= vis - n_last]
    rest = sorted((j for j in range(vis) if j not in must), key=lambda j: (-scores[j], j))
    return sorted((must + rest)[:k])


def attend_list(q, k, v, table, pos, page, pages, scale):
    """One token of one group: q [G, d], the listed pages, positions <= pos."""
    h_rows = [(p, o) for p in pages for o in range(page) if p * page + o <= pos]
    kr = np.array([k[table[p], o] for p, o in h_rows]).reshape(-1, q.shape[1])
    vr = np.array([v[table[p], o] for p, o in h_rows]).reshape(-1, q.shape[1])
    return softmax_rows(q, kr, vr, np.ones((q.shape[0], len(h_rows)), bool), scale)
