"""Softmax attention, its gradients and the pages of a cache in fp64 numpy and
plain lists.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).  Plain definitions of
include/kda_attn.h and include/kda_pages.h: one sequence and one head at a
time, one page at a time, no tiles and no fusion.

Shapes of one sequence: q [T, H, D], k, v [L, G, D]; query t has position
first + t, key j position j; `there` [L] marks keys that exist.
"""
from __future__ import annotations

import numpy as np


def _seen(T, L, first, causal, there):
    s = np.ones((T, L), bool) if there is None else np.tile(np.asarray(there, bool), (T, 1))
    if causal:
        s &= np.arange(L)[None, :] <= first + np.arange(T)[:, None]
    return s


def weights(q, k, h, scale, first=0, causal=True, there=None):
    """Softmax weights [T, L] of head h and lse [T]; rows that see nothing: 0 and -inf."""
    T, H, _ = q.shape
    L, G, _ = k.shape
    x = (np.asarray(q[:, h], np.float64) @ np.asarray(k[:, h // (H // G)], np.float64).T) * scale
    x = np.where(_seen(T, L, first, causal, there), x, -np.inf)
    P, lse = np.zeros((T, L)), np.full(T, -np.inf)
    for t in range(T):
        if L and np.isfinite(x[t].max()):
            m = x[t].max()
            e = np.exp(x[t] - m)
            P[t] = e / e.sum()
            lse[t] = m + np.log(e.sum())
    return P, lse


def attention(q, k, v, scale, first=0, causal=True, there=None):
    """Returns (o [T, H, D], lse [T, H])."""
    T, H, D = q.shape
    G = k.shape[1]
    o, lse = np.zeros((T, H, D)), np.zeros((T, H))
    for h in range(H):
        P, lse[:, h] = weights(q, k, h, scale, first, causal, there)
        vh = np.asarray(v[:, h // (H // G)], np.float64)
        o[:, h] = P @ (vh if there is None else np.where(np.asarray(there)[:, None], vh, 0.0))
    return o, lse


def attention_backward(q, k, v, gy, scale, causal=True):
    """Returns (gq, gk, gv) of whole sequences."""
    q, k, v, gy = (np.asarray(a, np.float64) for a in (q, k, v, gy))
    T, H, D = q.shape
    G = k.shape[1]
    gq, gk, gv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for h in range(H):
        g = h // (H // G)
        P, _ = weights(q, k, h, scale, 0, causal)
        gP = gy[:, h] @ v[:, g].T
        gS = P * (gP - (P * gP).sum(1, keepdims=True)) * scale
        gq[:, h] = gS @ k[:, g]
        gk[:, g] += gS.T @ q[:, h]
        gv[:, g] += P.T @ gy[:, h]
    return gq, gk, gv


# ---------------------------------------------------------- error bounds
#
# Of values that are computed from the given q, k, v in float32 with every
# weight (and score gradient) rounded to the operand type once: `half` is
# that rounding (0: none), u = 2^-24.  A dot product of n terms in any order
# is off by at most n u times the sum of its absolute terms.

U = 2.0 ** -24


def bounds(q, k, v, scale, half, first=0, causal=True, there=None):
    """Largest errors of o (before its own rounding) and lse."""
    T, H, D = q.shape
    L, G = k.shape[:2]
    eo, el = np.zeros((T, H, D)), np.zeros((T, H))
    for h in range(H):
        g = h // (H // G)
        P, lse = weights(q, k, h, scale, first, causal, there)
        # a score: D products and sums, the scale, its exponent's argument (values up to the score itself)
        mag = abs(scale) * (np.abs(q[:, h]) @ np.abs(k[:, g]).T)
        s = np.where(P > 0, mag, 0.0).max(1, initial=0.0) * (D + 8) * U
        rel = 2 * s + (L + 32) * U          # a weight: its exponential, the sum below it, rescaling
        vh = np.abs(v[:, g])
        eo[:, h] = (half + rel)[:, None] * (P @ (vh if there is None else np.where(np.asarray(there)[:, None], vh, 0.0)))
        el[:, h] = s + (np.where(np.isfinite(lse), np.abs(lse), 0.0) + L + 32) * U
    return eo, el


def backward_bounds(q, k, v, gy, scale, half, causal=True):
    """Largest errors of gq, gk, gv (before their own rounding); o is rounded by `half`, too."""
    T, H, D = q.shape
    G = k.shape[1]
    eq, ek, ev = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for h in range(H):
        g = h // (H // G)
        P, _ = weights(q, k, h, scale, 0, causal)
        o = P @ v[:, g]
        mag = abs(scale) * (np.abs(q[:, h]) @ np.abs(k[:, g]).T)
        s = np.where(P > 0, mag, 0.0).max(1, initial=0.0) * (D + 8) * U
        lse_err = s + (np.abs(np.log(np.maximum(P.max(1, initial=1e-30), 1e-30))) + T + 64) * U
        rel = (2 * s + lse_err + 64 * U)[:, None]
        gP = gy[:, h] @ v[:, g].T
        delta = (gy[:, h] * o).sum(1, keepdims=True)
        dmag = (np.abs(gy[:, h]) * np.abs(o)).sum(1, keepdims=True)
        pmag = np.abs(gy[:, h]) @ np.abs(v[:, g]).T
        # dS = P (gP - delta): its own rounding, o's in delta, and float32's in all of it
        eS = P * (half * (np.abs(gP - delta) + dmag) * 1.02 + (rel + (D + 8) * U) * (pmag + dmag))
        n = (T * (H // G) + 32) * U
        full = P * (np.abs(gP - delta) + half * dmag)
        eq[:, h] = abs(scale) * ((eS + n * full) @ np.abs(k[:, g]))
        ek[:, g] += abs(scale) * ((eS + n * full).T @ np.abs(q[:, h]))
        ev[:, g] += (P * (half + rel + n)).T @ np.abs(gy[:, h])
    return eq, ek, ev


# ----------------------------------------------------------------- pages

class Pool:
    """Tables, lengths and holders as lists; `data` [n_pages] holds anything."""

    def __init__(self, table, lengths, refs, page, data=None):
        self.table, self.lengths, self.refs, self.page = [list(r) for r in table], list(lengths), list(refs), page
        self.data = None if data is None else list(data)

    def used(self, length):
        return -(-length // self.page)

    def _clamp(self, x, slot):
        return max(0, min(x, len(self.table[slot]) * self.page))

    def _real(self, p):
        return 0 <= p < len(self.refs)

    def _free(self):
        return [p for p, r in enumerate(self.refs) if r <= 0]

    def resize(self, want):
        n = len(self.lengths)
        want = [self._clamp(w, s) for s, w in enumerate(want)]
        length = [self._clamp(w, s) for s, w in enumerate(self.lengths)]
        for s in range(n):
            for c in range(self.used(want[s]), self.used(length[s])):
                p = self.table[s][c]
                if self._real(p):
                    self.refs[p] -= 1
                self.table[s][c] = -1
        free, wanted, ok = self._free(), 0, []
        n_free = len(free)
        for s in range(n):
            need = max(0, self.used(want[s]) - self.used(length[s]))
            wanted += need
            ok.append(int(need == 0 or wanted <= n_free))
            if ok[s]:
                for c in range(self.used(length[s]), self.used(want[s])):
                    p = free.pop(0)
                    self.table[s][c] = p
                    self.refs[p] = 1
            self.lengths[s] = want[s] if ok[s] else length[s]
        return ok

    def fork(self, src, dst):
        slots = range(len(self.lengths))
        free = self._free()
        n_free, needed, ok, todo, taken = len(free), 0, [], [], set()
        for a, d in zip(src, dst):
            if a not in slots or d not in slots or d in taken:
                if d in slots:
                    taken.add(d)
                ok.append(0)
                continue
            taken.add(d)
            length = self._clamp(self.lengths[a], a)
            row = self.table[a][:self.used(length)]
            copy = a != d and length % self.page != 0 and self._real(row[-1])
            needed += copy
            ok.append(int(not copy or needed <= n_free))
            if ok[-1] and a != d:
                if copy:
                    todo.append((d, length, row[:-1], row[-1], free.pop(0)))
                else:
                    todo.append((d, length, row, None, None))
        old = {d: self.table[d][:self.used(self._clamp(self.lengths[d], d))] for d, *_ in todo}
        for d, length, row, tail, new in todo:
            for p in row:
                if self._real(p):
                    self.refs[p] += 1
            if tail is not None:
                self.refs[new] = 1
                if self.data is not None:
                    self.data[new] = self.data[tail]
        for d, length, row, tail, new in todo:
            for p in old[d]:
                if self._real(p):
                    self.refs[p] -= 1
            rest = max(len(old[d]), self.used(length))
            full = row + ([new] if tail is not None else [])
            self.table[d][:rest] = full + [-1] * (rest - len(full))
            self.lengths[d] = length
        return ok

    def compact(self):
        """Returns (table, refs, n_live); the data moves."""
        n_live = sum(r > 0 for r in self.refs)
        moves = [p for p in range(n_live, len(self.refs)) if self.refs[p] > 0]
        holes = [p for p in range(n_live) if self.refs[p] <= 0]
        to = dict(zip(moves, holes))
        refs = list(self.refs)
        for p, h in to.items():
            refs[h], refs[p] = self.refs[p], 0
            if self.data is not None:
                self.data[h] = self.data[p]
        table = [[to.get(p, p) if c < self.used(self._clamp(self.lengths[s], s)) else -1 for c, p in enumerate(row)]
                 for s, row in enumerate(self.table)]
        return table, refs, n_live
