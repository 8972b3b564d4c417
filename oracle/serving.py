"""Plain float64 forms of the HCA serving operators: norm with rotation, the
paged append, attention over paged entries, and the page operations on host
lists.  TEST INFRASTRUCTURE ONLY, like the rest of this package."""
from __future__ import annotations

import numpy as np

RUN = 16
EMPTY = -float(np.finfo(np.float32).max)


def norm_rope(x, pos, inv_freq=None, weight=None, eps=1e-6, norm=True, interleaved=True, inverse=False):
    """x [..., D] float64 at integer positions pos (broadcast over x's rows)."""
    y = np.array(x, np.float64)
    if norm:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
        if weight is not None:
            y = y * weight
    if inv_freq is None or len(inv_freq) == 0:
        return y
    h = len(inv_freq)
    r = y[..., -2 * h:]
    z = r[..., 0::2] + 1j * r[..., 1::2] if interleaved else r[..., :h] + 1j * r[..., h:]
    ang = np.asarray(pos, np.float64)[..., None] * inv_freq
    z = z * np.exp((-1j if inverse else 1j) * ang)
    if interleaved:
        r[..., 0::2], r[..., 1::2] = z.real, z.imag
    else:
        r[..., :h], r[..., h:] = z.real, z.imag
    return y


def gate_state(z, a):
    """(M, Z, A) of tokens z, a [n, D]; a gate of -inf drops its token."""
    D = z.shape[1]
    if not (z > -np.inf).any():
        return np.stack([np.full(D, EMPTY), np.zeros(D), np.zeros(D)])
    M = np.maximum(z.max(0), EMPTY)
    e = np.exp(z - M)
    return np.stack([M, e.sum(0), (e * np.where(e > 0, a, 0.0)).sum(0)])


def append(z, a, end, m):
    """Tokens z, a [end, D] of one sequence from position 0: the entries
    [end // m, D], and the open block's two parts [2, 3, D]."""
    entries = []
    for i in range(end // m):
        M, Z, A = gate_state(z[i * m:(i + 1) * m], a[i * m:(i + 1) * m])
        entries.append(np.where(Z == 0, 0.0, A / np.where(Z == 0, 1.0, Z)))
    lo = end // m * m
    mid = lo + (end - lo) // RUN * RUN
    D = z.shape[1]
    empty = np.stack([np.full(D, EMPTY), np.zeros(D), np.zeros(D)])
    parts = [gate_state(z[x:y], a[x:y]) if y > x else empty for x, y in ((lo, mid), (mid, end))]
    return np.array(entries).reshape(-1, D), np.stack(parts)


def attend(q, keys, sink, tau):
    """q [H, D] on keys [n, D] with sink [H] or None: out [H, D], lse [H], and the
    mean distance of the attended keys from the output, sum_j w_j |k_j - out|."""
    H, D = q.shape
    if len(keys) == 0:
        return np.zeros((H, D)), np.full(H, -np.inf), np.zeros((H, D))
    lg = q @ keys.T * tau
    mx = lg.max(1)
    sg = np.full(H, -np.inf) if sink is None else sink
    M = np.maximum(mx, sg)
    w = np.exp(lg - M[:, None])
    den = w.sum(1) + np.exp(sg - M)
    w = w / den[:, None]
    out = w @ keys
    spread = np.stack([(w[h][:, None] * np.abs(keys - out[h])).sum(0) for h in range(H)])
    with np.errstate(divide="ignore"):
        lse = mx + np.log(np.exp(lg - mx[:, None]).sum(1))
    return out, lse, spread


class Pages:
    """The page operations on host lists: rows of page ids, and page contents."""

    def __init__(self, N, P, R, max_pages, pool):
        self.N, self.P, self.max_pages = N, P, max_pages
        self.rows = [[] for _ in range(R)]
        self.ref = [0] * N
        self.pool = pool          # [L, N, P, D] array

    def _take(self, k):
        free = [i for i in range(self.N) if self.ref[i] == 0]
        if len(free) < k:
            raise MemoryError
        return free[:k]

    def reserve(self, rows, n):
        need = [max(0, -(-e // self.P) - len(self.rows[r])) for r, e in zip(rows, n)]
        new = self._take(sum(need))
        for r, k in zip(rows, need):
            for _ in range(k):
                self.rows[r].append(new.pop(0))
                self.ref[self.rows[r][-1]] = 1

    def fork(self, src, dst, n):
        new = self._take(sum(e % self.P != 0 for e in n))
        for s, d, e in zip(src, dst, n):
            assert not self.rows[d]
            self.rows[d] = self.rows[s][:e // self.P]
            for p in self.rows[d]:
                self.ref[p] += 1
        for s, d, e in zip(src, dst, n):
            if e % self.P:
                p = new.pop(0)
                self.pool[:, p, :e % self.P] = self.pool[:, self.rows[s][e // self.P], :e % self.P]
                self.ref[p] = 1
                self.rows[d].append(p)

    def free(self, rows):
        for r in rows:
            for p in self.rows[r]:
                self.ref[p] -= 1
            self.rows[r] = []

    def compact(self):
        live = sum(r > 0 for r in self.ref)
        holes = [i for i in range(live) if self.ref[i] == 0]
        new = {i: i for i in range(self.N)}
        for i in range(live, self.N):
            if self.ref[i] > 0:
                new[i] = holes.pop(0)
                self.pool[:, new[i]] = self.pool[:, i]
                self.ref[new[i]], self.ref[i] = self.ref[i], 0
        self.rows = [[new[p] for p in r] for r in self.rows]
        return live

    def table(self):
        t = np.full((len(self.rows), self.max_pages), -1, np.int32)
        for i, r in enumerate(self.rows):
            t[i, :len(r)] = r
        return t
