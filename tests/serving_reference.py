"""Plain 64-bit implementations of the serving operators for the tests: attention through a
page table, the page operations on host lists, sampled verification. Written from the
operators' definitions; they share no code with the library."""
from __future__ import annotations

import numpy as np
import torch

D = 128


def gather(pages, row, n):
    """Tokens 0 .. n - 1 of a sequence, float64 [n, kv heads, D] on the host."""
    ps = pages.shape[2]
    need = -(-n // ps)
    x = pages[row[:need].long()].transpose(1, 2).reshape(-1, pages.shape[1], D)[:n]
    return x.double().cpu()


def attend(q, k, v, seen, scale):
    """q [Hq, D], k / v [n, Hkv, D], the first `seen` keys visible. Returns (out [Hq, D], the error
    scales: sum p |v| [Hq, D], the largest |v| seen, the largest sum |q| |k| * scale)."""
    hq, hkv = q.shape[0], k.shape[1]
    rep = hq // hkv
    if seen <= 0:
        z = torch.zeros((hq, D), dtype=torch.float64)
        return z, z, 0.0, 0.0
    k, v = k[:seen], v[:seen]
    s = torch.einsum("hrd,nhd->hrn", q.view(hkv, rep, D), k) * scale
    p = torch.softmax(s, -1)
    out = torch.einsum("hrn,nhd->hrd", p, v).reshape(hq, D)
    mag = torch.einsum("hrn,nhd->hrd", p, v.abs()).reshape(hq, D)
    dot = torch.einsum("hrd,nhd->hrn", q.view(hkv, rep, D).abs(), k.abs()).max() * abs(scale)
    return out, mag, float(v.abs().max()), float(dot)


def attention_bound(out, mag, vmax, dot, n, bf16):
    """How far a right kernel may be from `attend`, element by element.

    Scores: bf16 products are exact in f32 and their sums of 128 (in any order, f32) are off by at most
    128 * 2^-24 = 2^-17 of sum |q| |k|; an f32 q enters as bf16 hi + lo, off by 2^-8 * 2^-8 = 2^-16 of it, and its
    scaling by 2^-24. So a score is off by d = dot * (2^-17 + 2^-16 + 2^-23) < dot * 2^-15, a weight by
    e^(2 d) - 1 < 2.1 d of itself (its own score's error and the sum's), plus its exponential (2^-21 of itself with the
    argument's rounding at |s| < 8 log2 units) and its own rounding: bf16 2^-8, or hi + lo 2^-16. Sums over n keys in
    f32: at most n 2^-24 of sum p |v| (numerator) and of 1 (denominator). The result's rounding: 2^-8 or 2^-24."""
    d = dot * 2.0 ** -15
    w = 2.1 * d + 2.0 ** -20 + (2.0 ** -8 if bf16 else 2.0 ** -16) + 2 * n * 2.0 ** -24 + 2.0 ** -20
    return w * mag + (w - (2.0 ** -8 if bf16 else 2.0 ** -16)) * out.abs() + (2.0 ** -8 if bf16 else 2.0 ** -23) * out.abs() + 1e-30


class Pages:
    """The page operations on host lists; `k` holds one value per (page, slot) standing for its contents."""

    def __init__(self, n_pages, ps, max_seqs, max_pages):
        self.ps, self.max_pages = ps, max_pages
        self.table = [[] for _ in range(max_seqs)]
        self.lens = [0] * max_seqs
        self.refs = [0] * n_pages
        self.copies = []

    def _take(self):
        p = self.refs.index(0)
        self.refs[p] = 1
        return p

    def fork(self, parents, children):
        n = len(self.lens)
        if len(set(children)) != len(children):
            return False
        for a, c in zip(parents, children):
            if not (0 <= a < n and 0 <= c < n and a != c) or self.lens[c]:
                return False
        old = [(list(self.table[a]), self.lens[a]) for a in parents]
        for (row, length), c in zip(old, children):
            self.table[c], self.lens[c] = list(row), length
            for p in row:
                self.refs[p] += 1
        return True

    def extend(self, n_new):
        before = ([list(r) for r in self.table], list(self.lens), list(self.refs))
        copies = []
        for s, n in enumerate(n_new):
            if n <= 0:
                continue
            ok = self.lens[s] + n <= self.max_pages * self.ps
            if ok and self.lens[s] % self.ps and self.refs[self.table[s][-1]] > 1:
                ok = 0 in self.refs
                if ok:
                    a = self.table[s][-1]
                    b = self._take()
                    self.refs[a] -= 1
                    self.table[s][-1] = b
                    copies.append((a, b))
            self.lens[s] += n
            while ok and len(self.table[s]) * self.ps < self.lens[s]:
                ok = 0 in self.refs
                if ok:
                    self.table[s].append(self._take())
            if not ok:
                self.table, self.lens, self.refs = before
                return False
        self.copies += copies
        return True

    def trim(self, new_lens):
        for s, n in enumerate(new_lens):
            if 0 <= n < self.lens[s]:
                while len(self.table[s]) > -(-n // self.ps):
                    self.refs[self.table[s].pop()] -= 1
                self.lens[s] = n

    def compact(self):
        live = sum(n > 0 for n in self.refs)
        free = [p for p in range(live) if not self.refs[p]]
        to = {}
        for p in range(live, len(self.refs)):
            if self.refs[p]:
                to[p] = free.pop(0)
                self.refs[to[p]], self.refs[p] = self.refs[p], 0
                self.copies.append((p, to[p]))
        self.table = [[to.get(p, p) for p in r] for r in self.table]
        return live

    def arrays(self):
        t = np.full((len(self.lens), self.max_pages), -1, np.int32)
        for s, r in enumerate(self.table):
            t[s, :len(r)] = r
        return t, np.array(self.lens, np.int32), np.array(self.refs, np.int32)


def verify(p, q, draft, u, n_draft):
    """One sequence: p [k, V], q [k - 1, V], draft [k - 1], u [k] (float64 arrays) -> (accepted, next token)."""
    V = p.shape[1]
    m = 0
    while m < n_draft and 0 <= draft[m] < V and u[m] * q[m, draft[m]] < p[m, draft[m]]:
        m += 1

    def mass(x):
        return np.where(np.isfinite(x) & (x > 0), x, 0.0)

    with np.errstate(invalid="ignore"):
        r = mass(p[m] - q[m]) if m < n_draft else mass(p[m])
    if not r.any():
        r = mass(p[m])
    if not r.any():
        return m, 0
    c = np.cumsum(r)
    over = np.nonzero(c > u[-1] * c[-1])[0]
    return m, int(over[0] if len(over) else np.nonzero(r)[0][-1])
