"""Oracles of the shared pages of a cache and of the norms around a block (NumPy).

``Pool`` follows the calls one item at a time. ``norm`` computes in 64 bits and
also returns how far fp32 arithmetic may be off, from rounding errors alone.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24          # half a step of fp32, relative
BAD_PAGE, BAD_ROW, NO_PAGE = 0x40, 0x80, 0x100


class Pool:
    """table [rows, width], held [rows], refs [pages] and caches [pages, bytes]
    as arrays that the calls change in place; each returns its flags."""

    def __init__(self, table, held, refs, page_size, caches=()):
        self.table, self.held, self.refs = table.copy(), held.copy(), refs.copy()
        self.ps, self.caches = page_size, [c.copy() for c in caches]

    def _entries(self, tokens):
        return -(-int(tokens) // self.ps)

    def _row_ok(self, r):
        return 0 <= r < len(self.held)

    def _page_ok(self, p):
        return 0 <= p < len(self.refs)

    def _count_ok(self, r):
        """Whether a row holds as many entries as it may have."""
        return 0 <= self.held[r] <= self.table.shape[1]

    def _drop(self, p):
        if self.refs[p] > 0:
            self.refs[p] -= 1
            return 0
        return BAD_PAGE

    def fork(self, parents, children, tokens):
        flags, held = 0, self.held.copy()
        for i, (p, c, t) in enumerate(zip(parents, children, tokens)):
            ok = self._row_ok(p) and self._row_ok(c) and 0 <= t <= self.table.shape[1] * self.ps
            ok = ok and c not in children[:i] and p not in children
            ok = ok and held[c] == 0 and self._entries(t) <= held[p] <= self.table.shape[1]
            if not ok:
                flags |= BAD_ROW
                continue
            n = self._entries(t)
            for e in range(n):
                self.table[c, e] = page = self.table[p, e]
                if self._page_ok(page):
                    self.refs[page] += 1
                else:
                    flags |= BAD_PAGE
            self.held[c] = n
        return flags

    def release(self, rows, keep):
        flags = 0
        for r, k in zip(rows, keep):
            if not self._row_ok(r) or k < 0 or not self._count_ok(r):
                flags |= BAD_ROW
                continue
            left = min(self._entries(k), self.table.shape[1])
            for e in range(left, self.held[r]):
                page, self.table[r, e] = self.table[r, e], -1
                flags |= self._drop(page) if self._page_ok(page) else BAD_PAGE
            self.held[r] = min(self.held[r], left)
        return flags

    def reserve(self, rows, start, end):
        flags = 0
        refs, held = self.refs.copy(), self.held.copy()      # as found
        free = list(np.flatnonzero(refs == 0))
        at, full = 0, False
        copies, dropped = [], []
        for i, (r, a, b) in enumerate(zip(rows, start, end)):
            if (not self._row_ok(r) or r in rows[:i] or not 0 <= a <= b <= self.table.shape[1] * self.ps
                    or not self._count_ok(r)):
                flags |= BAD_ROW
                continue
            lo, hi = (a // self.ps if a < b else self._entries(b)), self._entries(b)
            own = []
            for e in range(lo, min(hi, held[r])):
                page = self.table[r, e]
                if not self._page_ok(page):
                    flags |= BAD_PAGE
                    if -1 - len(refs) <= page <= -2:
                        self.table[r, e] = -1
                elif refs[page] > 1:
                    own.append(e)
            places = own + list(range(held[r], hi))
            full = full or (bool(places) and at + len(places) > len(free))
            if not places:
                continue
            if full:
                flags |= NO_PAGE
                continue
            for e in places:
                page, at = free[at], at + 1
                if e in own:
                    dropped.append(self.table[r, e])
                    if e == lo and a % self.ps:
                        copies.append((self.table[r, e], page))
                self.table[r, e] = page
                self.refs[page] = 1
            self.held[r] = max(held[r], hi)
        for p in dropped:
            flags |= self._drop(p)
        for c in self.caches:
            for s, d in copies:
                c[d] = c[s]
        return flags

    def compact(self):
        used = np.flatnonzero(self.refs != 0)
        n = len(used)
        src, dst = used[used >= n], np.flatnonzero(self.refs[:n] == 0)
        to = np.arange(len(self.refs))
        to[src] = dst
        for c in self.caches:
            c[dst] = c[src]
        self.refs[dst] = self.refs[src]
        self.refs[src] = 0
        flags = 0
        was = np.zeros(len(self.refs), bool)
        was[used] = True
        for r, h in enumerate(self.held):
            if not self._count_ok(r):
                flags |= BAD_ROW
            for e in range(min(h, self.table.shape[1])):
                p = self.table[r, e]
                if not self._page_ok(p) or (p >= n and not was[p]):
                    flags |= BAD_PAGE
                else:
                    self.table[r, e] = to[p]
        return n, flags


def norm(x, y=None, post=False, post_w=None, post_b=None, gate=None, sigmoid=False, pre_w=None,
         pre_b=None, layer=False, scale=1.0, offset=0.0, eps=1e-6):
    """(r, h, bound on |r - fp32's r|, bound on |h - fp32's h|), before the
    outputs' own rounding. Sums of H terms are made of at most 16 per thread and
    ten more over threads: 27 roundings of what is summed in magnitude, and the
    mean's product."""
    def normed(v, dv, w, b):
        dm, m = 0.0, 0.0
        if layer:
            m = v.mean(-1, keepdims=True)
            dm = 28 * U * np.abs(v).mean(-1, keepdims=True) + dv.mean(-1, keepdims=True)
        c = v - m
        dc = dv + dm + U * np.abs(c)
        std = np.sqrt((c * c).mean(-1, keepdims=True) + eps)
        # the root of a mean of squares moves by at most the root mean square of
        # its terms' errors; sum, product, eps, root and quotient round themselves
        ds = np.sqrt((dc * dc).mean(-1, keepdims=True)) / std + (28 / 2 + 4) * U
        w1 = np.ones(v.shape[-1]) if w is None else w + offset
        out = c / std * w1
        d = dc / std * np.abs(w1) + np.abs(out) * (ds + 3 * U) * 1.01
        if b is not None:
            out = out + b
            d = d + U * np.abs(out)
        return out, d

    x = np.asarray(x, np.float64)
    r, dr = x, np.zeros_like(x)
    if y is not None:
        u = np.asarray(y, np.float64)
        du = np.zeros_like(u)
        if post:
            u, du = normed(u, du, post_w, post_b)
        g, dg = np.ones_like(u), 0.0
        if gate is not None:
            g = np.broadcast_to(np.asarray(gate, np.float64), u.shape)
            if sigmoid:      # exp, one more, quotient: 2, 1 and 2 half steps
                with np.errstate(over="ignore"):
                    g = 1.0 / (1.0 + np.exp(-g))
                dg = 8 * U * g + 2.0 ** -126
        add = scale * g * u
        r = x + add
        dr = np.abs(scale) * (np.abs(g) * du + dg * np.abs(u)) + 3 * U * np.abs(add) + U * np.abs(r)
    h, dh = normed(r, dr, pre_w, pre_b)
    return r, h, dr, dh
