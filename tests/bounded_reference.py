"""Plain 64-bit implementations of the operators that fill and bound the cache, for the tests: norms and
rotation of rows, attention that sees a window and a few first tokens, the weights it gives, eviction. Written
from the operators' definitions; they share no code with the library."""
from __future__ import annotations

import numpy as np
import torch

D = 128


def bf16_steps(x):
    """x (float64) rounded to bf16, and how far it lies from a border between two roundings, relative to itself."""
    m, e = torch.frexp(x)
    t = m.abs() * 2 ** 8                      # a unit is a step of bf16
    f = t - t.floor()
    return torch.copysign(torch.ldexp(torch.round(t), e - 8), x), (f - 0.5).abs() / t.clamp(min=1e-300)


def norm_rope(x, w, cs, eps, cast):
    """x float64 [heads, D], w [D], cs [D / 2, 2]. Returns (y [heads, D], the size |a c| + |b s| of each value's terms,
    the least distance of a rounding on the way from its border)."""
    inv = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / D + eps)
    y, far = x * inv, torch.ones_like(x)
    if cast:
        y, f1 = bf16_steps(y)
        y, f2 = bf16_steps(y * w)
        far = torch.minimum(f1, f2)
    else:
        y = y * w
    a, b, c, s = y[:, :D // 2], y[:, D // 2:], cs[:, 0], cs[:, 1]
    far = torch.minimum(far[:, :D // 2], far[:, D // 2:])
    return (torch.cat([a * c - b * s, b * c + a * s], 1), torch.cat([(a * c).abs() + (b * s).abs(),
                                                                    (b * c).abs() + (a * s).abs()], 1),
            torch.cat([far, far], 1))


def visible(p, n, window, sinks):
    """Which of the keys 0 .. n - 1 the row at slot p sees."""
    t = torch.arange(n)
    return (t <= p) & ((t > p - window) | (t < sinks))


def attend(q, k, v, see, scale):
    """q [Hq, D], k, v [n, Hkv, D], see [n]: (out, weights summed over a kv head's q heads [Hkv, n], sum p |v|, the
    largest scale * sum |q| |k|), float64. A row that sees nothing gives 0."""
    hq, hkv = q.shape[0], k.shape[1]
    if not bool(see.any()):
        z = torch.zeros((hq, D), dtype=torch.float64)
        return z, torch.zeros((hkv, k.shape[0]), dtype=torch.float64), z, 0.0
    qq = q.view(hkv, hq // hkv, D)
    kk, vv = k[see], v[see]
    p = torch.softmax(torch.einsum("hrd,nhd->hrn", qq, kk) * scale, -1)
    out = torch.einsum("hrn,nhd->hrd", p, vv).reshape(hq, D)
    mag = torch.einsum("hrn,nhd->hrd", p, vv.abs()).reshape(hq, D)
    w = torch.zeros((hkv, k.shape[0]), dtype=torch.float64)
    w[:, see] = p.sum(1)
    dot = float(torch.einsum("hrd,nhd->hrn", qq.abs(), kk.abs()).max()) * abs(scale)
    return out, w, mag, dot


def weight_bound(dot, n):
    """How far a weight of a right kernel may be off, relative to itself: its score, an f32 sum of 128 exact
    products (or of the three parts of an f32 q, whose rest is below 2^-24) is off by at most d = 2^-17 + 2^-23 of
    the sum of their magnitudes, and so is the largest one; the sum of n weights by n 2^-24, and it carries the
    scores' errors again; each exponential by 2^-21 (its argument rounded in units of up to 2^6) and the division
    and the sum over a few heads by 2^-22."""
    d = dot * (2.0 ** -17 + 2.0 ** -23)
    return 2.1 * d + n * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -21


def evict(weights, n, keep, sinks, recent):
    """The tokens that stay of n: weights [n] float64."""
    if keep < 0 or keep >= n:
        return np.arange(n)
    first = min(sinks, keep)
    last = min(recent, keep - first)
    middle = np.arange(first, n - last)
    w = np.where(np.isnan(weights[middle]), -np.inf, weights[middle])
    best = middle[np.lexsort((middle, -w))][:keep - first - last]
    return np.sort(np.concatenate([np.arange(first), best, np.arange(n - last, n)]))


def make_cache(g, lens, hkv, ps, spare=3, room=0):
    """Random bf16 caches and the page table (pages in random order, -1 past the end) of sequences of these lengths;
    room: tokens of the table beyond the longest."""
    need = [max(0, -(-n // ps)) for n in lens]
    width, used, n_pages = max(1, -(-(max(lens) + room) // ps)), 0, sum(need) + spare
    perm = torch.randperm(n_pages, generator=g, device=g.device).tolist()
    table = []
    for n in need:
        table.append([perm[used + i] for i in range(n)] + [-1] * (width - n))
        used += n
    shape = (n_pages, hkv, ps, D)
    kp = torch.randn(shape, generator=g, device=g.device).to(torch.bfloat16)
    vp = torch.randn(shape, generator=g, device=g.device).to(torch.bfloat16)
    return kp, vp, torch.tensor(table, dtype=torch.int32, device=g.device)


def tokens(pages, row, n):
    """Tokens 0 .. n - 1 of a sequence, float64 [n, kv heads, D] on the host."""
    ps = pages.shape[2]
    x = pages[row[:-(-n // ps)].long()].transpose(1, 2).reshape(-1, pages.shape[1], D)[:n]
    return x.double().cpu()


def out_bound(out, mag, dot, n, bf16, parts):
    """How far a row of a right kernel may be from `attend`: its weights' errors (weight_bound, and their own entry
    into the products: bf16 2^-8 in one part, 2^-16 in two, 2^-24 in three) count with sum p |v|, the sum over n keys
    in f32 with n 2^-24 of that; the result is rounded to its type."""
    w = weight_bound(dot, n) + 2.0 ** -(8 * parts) + n * 2.0 ** -24
    return w * mag + out.abs() * (2.0 ** -8 if bf16 else 2.0 ** -23) + 1e-30
