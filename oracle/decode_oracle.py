"""fp64 oracle of the decode step: paged cache, per-head norms and rotation,
attention of drafted trees, verification of drafted tokens.

TEST INFRASTRUCTURE ONLY, like ivc_oracle. Plain definitions in numpy float64
and Python integers, one sequence, head and node at a time.
"""
from __future__ import annotations

import numpy as np


class PagedCache:
    """The cache as plain arrays; every operation as include/ivc.h states it.
    An operation that is refused raises ValueError("bad" or "full") and changes
    nothing."""

    def __init__(self, layers, pages, kv_heads, page_tokens, head_dim, max_seqs, max_pages):
        shape = (layers, pages, kv_heads, page_tokens, head_dim)
        self.k, self.v = np.zeros(shape), np.zeros(shape)
        self.pt = page_tokens
        self.table = np.full((max_seqs, max_pages), -1, dtype=np.int32)
        self.length = np.zeros(max_seqs, dtype=np.int32)
        self.n_pages = np.zeros(max_seqs, dtype=np.int32)
        self.ref = np.zeros(pages, dtype=np.int32)
        self.free = [pages - 1 - i for i in range(pages)]  # the last one is taken next

    def _named(self, seqs):
        seqs = [int(s) for s in seqs]
        if len(set(seqs)) != len(seqs) or any(s < 0 or s >= len(self.length) for s in seqs):
            raise ValueError("bad")
        return seqs

    def _take(self, s, n):
        for _ in range(n):
            p = self.free.pop()
            self.ref[p] = 1
            self.table[s, self.n_pages[s]] = p
            self.n_pages[s] += 1

    def _release(self, pages):
        gone = []
        for p in pages:
            self.ref[p] -= 1
            if self.ref[p] == 0:
                gone.append(p)
        self.free.extend(sorted(gone, reverse=True))

    def reserve(self, tokens, seqs):
        seqs = self._named(seqs)
        if any(t < 0 for t in tokens):
            raise ValueError("bad")
        want = [-(-(int(self.length[s]) + int(t)) // self.pt) for s, t in zip(seqs, tokens)]
        need = [max(0, w - int(self.n_pages[s])) for s, w in zip(seqs, want)]
        if any(w > self.table.shape[1] for w in want) or sum(need) > len(self.free):
            raise ValueError("full")
        for s, m in zip(seqs, need):
            self._take(s, m)

    def fork(self, src, dst, share):
        dst = self._named(dst)
        if any(s < 0 or s >= len(self.length) for s in src):
            raise ValueError("bad")
        if any(self.length[d] or self.n_pages[d] for d in dst):
            raise ValueError("bad")
        lens = [int(self.length[s]) for s in src]
        full = [n // self.pt if share else 0 for n in lens]
        need = [-(-n // self.pt) - f for n, f in zip(lens, full)]
        if sum(need) > len(self.free):
            raise ValueError("full")
        for s, d, n, f, m in zip(src, dst, lens, full, need):
            self.table[d, :f] = self.table[s, :f]
            self.ref[self.table[d, :f]] += 1
            self.n_pages[d], self.length[d] = f, n
            self._take(d, m)
            for t in range(f * self.pt, n):
                self._copy(s, t, d, t)

    def _slot(self, s, t):
        return int(self.table[s, t // self.pt]), t % self.pt

    def _copy(self, s, t, d, u):
        (p, i), (q, j) = self._slot(s, t), self._slot(d, u)
        for x in (self.k, self.v):
            x[:, q, :, j] = x[:, p, :, i]

    def compact(self, count, keep=None, start=None, seqs=None):
        seqs = self._named(range(len(count)) if seqs is None else seqs)
        start = [int(self.length[s]) for s in seqs] if start is None else [int(a) for a in start]
        plans = []
        for i, (s, a, m) in enumerate(zip(seqs, start, count)):
            cap = int(self.n_pages[s]) * self.pt
            if not 0 <= a <= self.length[s] or m < 0 or a + m > cap:
                raise ValueError("bad")
            kept = list(range(m)) if keep is None else [int(x) for x in keep[i][:m]]
            if len(kept) != m or any(x < 0 or a + x >= cap for x in kept) or \
                    any(y <= x for x, y in zip(kept, kept[1:])):
                raise ValueError("bad")
            moves = [(a + x, a + j) for j, x in enumerate(kept) if x != j]
            if any(self.ref[self._slot(s, u)[0]] != 1 for _, u in moves):
                raise ValueError("bad")
            if (a + m) % self.pt and self.ref[self._slot(s, a + m)[0]] != 1:
                raise ValueError("bad")
            plans.append((s, a + m, moves))
        gone = []
        for s, n, moves in plans:
            for t, u in moves:
                self._copy(s, t, s, u)
            left = -(-n // self.pt)
            gone += [int(p) for p in self.table[s, left:self.n_pages[s]]]
            self.table[s, left:] = -1
            self.length[s], self.n_pages[s] = n, min(left, self.n_pages[s])
        self._release(gone)

    def drop(self, seqs):
        seqs = self._named(seqs)
        gone = []
        for s in seqs:
            gone += [int(p) for p in self.table[s, :self.n_pages[s]]]
            self.table[s] = -1
            self.length[s] = self.n_pages[s] = 0
        self._release(gone)

    def tokens(self, s, n, layer):
        """Keys and values of the first n tokens of sequence s: [n, heads, D]."""
        slots = [self._slot(s, t) for t in range(n)]
        return tuple(np.stack([x[layer, p, :, i] for p, i in slots]) if slots else
                     np.zeros((0,) + x.shape[2:3] + x.shape[4:]) for x in (self.k, self.v))


def norm_rope(x, gamma, positions, theta, eps):
    """Per-head norm and rotation of x [N, heads, D] (gamma None: as it is)."""
    N, H, D = x.shape
    out = np.empty_like(x)
    for n in range(N):
        for h in range(H):
            y = x[n, h] / np.sqrt(np.mean(x[n, h] ** 2) + eps) * gamma
            for j in range(D // 2):
                t = float(positions[n]) * theta ** (-2.0 * j / D)
                out[n, h, j] = y[j] * np.cos(t) - y[j + D // 2] * np.sin(t)
                out[n, h, j + D // 2] = y[j + D // 2] * np.cos(t) + y[j] * np.sin(t)
    return out


def ancestors(parents, i):
    """Node i and its ancestors."""
    got = []
    while i >= 0:
        got.append(i)
        i = int(parents[i])
    return got


def tree_attend(q, k, v, length, parents, scale):
    """q [n, q_heads, D]; k, v [length + n, kv_heads, D] in float64."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = np.empty_like(q)
    for i in range(n):
        seen = list(range(length)) + sorted(length + a for a in ancestors(parents, i))
        for h in range(Hq):
            s = k[seen, h // G] @ q[i, h] * scale
            w = np.exp(s - s.max())
            out[i, h] = (w / w.sum()) @ v[seen, h // G]
    return out


def verify(p, q, tokens, parents, u, u_next):
    """One tree: (path, next token or -1). p, q float64 [n, V] (q None: drafts not
    drawn at random)."""
    p = np.where(p > 0, p, 0.0)
    q = None if q is None else np.where(q > 0, q, 0.0)
    cur, path = 0, [0]
    r, z, w = p[0].copy(), 1.0, 1.0
    d = None if q is None else q[0].copy()
    for j in range(1, len(tokens)):
        c = int(tokens[j])
        if parents[j] != cur or not z > 0:
            continue
        qc = 1.0 if q is None else d[c]
        if u[j] * qc * z < r[c] * w:
            cur = j
            path.append(j)
            r, z, w = p[j].copy(), 1.0, 1.0
            d = None if q is None else q[j].copy()
        elif q is None:
            z -= r[c]
            r[c] = 0.0
        else:
            r = np.maximum(r * (1.0 / z) - d * (1.0 / w if w > 0 else 0.0), 0.0)
            z = r.sum()
            w -= qc
            d[c] = 0.0
    if not r.sum() > 0:
        r = p[cur]
    total = np.cumsum(r)
    if not (total[-1] > 0 and np.isfinite(total[-1])):
        return path, -1
    over = np.nonzero((total > u_next * total[-1]) & (r > 0))[0]
    return path, int(over[0] if len(over) else np.nonzero(r > 0)[0][-1])
