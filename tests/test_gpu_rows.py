"""Norms and rotation of packed rows with their cache write, on the GPU against a plain 64-bit implementation."""
import math

import numpy as np
import pytest
import torch

import bounded_reference as ref
from transformer_decode_step_weight_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = 128


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Case:
    def __init__(self, rows, lens, hq, hkv, ps, dtype, seed=0, scale=1.0):
        g = _gen(seed)
        need = [-(-n // ps) for n in lens]
        used, n_pages = 0, sum(need) + 3
        perm = torch.randperm(n_pages, generator=g, device=DEV).tolist()
        width = max(1, max(need))
        table = []
        for n in need:
            table.append([perm[used + i] for i in range(n)] + [-1] * (width - n))
            used += n
        self.rows, self.lens, self.hq, self.hkv, self.ps = rows, lens, hq, hkv, ps
        self.cu = [0]
        for n in rows:
            self.cu.append(self.cu[-1] + n)
        self.table = _ints(table)
        self.k = torch.randn((n_pages, hkv, ps, D), generator=g, device=DEV).to(torch.bfloat16)
        self.v = torch.randn((n_pages, hkv, ps, D), generator=g, device=DEV).to(torch.bfloat16)
        self.x = (torch.randn((self.cu[-1], (hq + 2 * hkv) * D), generator=g, device=DEV) * scale).to(dtype)
        self.qn = (1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16)
        self.kn = (1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16)
        self.rope = api.rope_table(max(max(lens), 1) + 70, D, 1e6, DEV)
        self.slots = [m - n + j for n, m in zip(rows, lens) for j in range(n)]
        self.seqs = [b for b, n in enumerate(rows) for _ in range(n)]

    def call(self, **kw):
        x, cu, lens, eps = (kw.pop(a, None) for a in ("x", "cu", "lens", "eps"))
        return api.qk_norm_rope(self.x if x is None else x, self.qn, self.kn, self.rope, self.k, self.v, self.table,
                                _ints(self.cu) if cu is None else cu, _ints(self.lens) if lens is None else lens,
                                1e-6 if eps is None else eps, **kw)

    def check(self, q, k0, v0, cast=False, positions=None, axes=None, eps=1e-6, pick=None, off=0):
        """q and the caches against the 64-bit form; cache slots of no row are as in k0, v0.

        A sum of 128 squares in f32 is off by 128 2^-24 of itself, its root by half of that: 2^-18; the division,
        the products and the difference of two terms by 8 2^-24 of the terms; the result is rounded to its type. With
        `cast` a value that lies within 2^-15 of itself of a border may go to the other side of it, a step of 2^-7 of
        itself at each of the two roundings."""
        x, rope = self.x.double().cpu(), self.rope.double().cpu()
        k, v, want_k, want_v = (t.double().cpu() for t in (self.k, self.v, k0, v0))
        q, tb, hq, hkv = q.double().cpu(), self.table.cpu(), self.hq, self.hkv
        half = 2.0 ** -8 if self.out_bf16 else 2.0 ** -24
        ax = torch.zeros(64, dtype=torch.long) if axes is None else torch.tensor(list(axes))
        i = torch.arange(64)
        near = total = 0
        for r in range(len(self.slots)) if pick is None else pick:
            b, slot = self.seqs[r], self.slots[r]
            pos = torch.full((4,), slot) if positions is None else positions[:, r].long().cpu()
            cs = rope[pos[ax], i]
            heads = x[off + r].view(-1, D)
            page = int(tb[b, slot // self.ps])
            for lo, hi, w, got, rnd in ((0, hq, self.qn, q[off + r], half),
                                        (hq, hq + hkv, self.kn, k[page, :, slot % self.ps], 2.0 ** -8)):
                want, size, far = ref.norm_rope(heads[lo:hi], w.double().cpu(), cs, eps, cast)
                tol = size * (2.0 ** -18 + 8 * 2.0 ** -24) + want.abs() * rnd * 1.01 + 1e-30
                tie = far < 2.0 ** -15
                tol = torch.where(tie, tol + 2.02 * 2.0 ** -7 * size, tol)
                assert bool(((got - want).abs() <= tol).all()), (r, lo, float(((got - want).abs() / tol).max()))
                near, total = near + int(tie.sum()), total + tie.numel()
            assert torch.equal(v[page, :, slot % self.ps], heads[hq + hkv:].to(torch.bfloat16).double()), r
            want_k[page, :, slot % self.ps] = k[page, :, slot % self.ps]
            want_v[page, :, slot % self.ps] = v[page, :, slot % self.ps]
        if pick is None:   # nothing else in the caches has changed
            assert torch.equal(k, want_k) and torch.equal(v, want_v)
        # a rounding lies within 2^-15 of its value of a border in 1.2 % of all cases (values of 128 .. 256 steps), a
        # product of two bf16 values on it in 0.4 %, and a rotated value comes from four: the allowance above is rare
        assert near <= 0.2 * total
        assert api.check_device_error() == 0

    out_bf16 = False


CASES = [([1], [1], 4, 2, 16), ([1, 1, 1], [1, 17, 300], 8, 8, 16), ([5], [9], 1, 1, 16), ([128], [128], 4, 4, 16),
         ([129, 0, 127], [129, 40, 200], 4, 2, 32), ([3, 31], [1000, 331], 32, 8, 16), ([33, 70], [129, 70], 12, 4, 7),
         ([0, 0, 2, 0], [5, 0, 2, 0], 5, 1, 24), ([1] * 70, list(range(1, 141, 2)), 8, 2, 16)]


@pytest.mark.parametrize("src,dst", [(torch.float32, torch.float32), (torch.float32, torch.bfloat16),
                                     (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("cast", [False, True])
@pytest.mark.parametrize("rows,lens,hq,hkv,ps", CASES)
def test_rows(cuda_lib, rows, lens, hq, hkv, ps, cast, src, dst):
    c = Case(rows, lens, hq, hkv, ps, src, seed=sum(rows) + hq, scale=1.5)
    k0, v0 = c.k.clone(), c.v.clone()
    c.out_bf16 = dst == torch.bfloat16
    q = c.call(cast=cast, dtype=dst)
    assert q.dtype == dst and q.shape == (c.cu[-1], hq, D)
    c.check(q, k0, v0, cast=cast)


@pytest.mark.parametrize("n_axes", [1, 2, 3, 4])
def test_rows_positions_of_several_axes(cuda_lib, n_axes):
    c = Case([40, 9], [70, 9], 4, 2, 16, torch.float32, seed=n_axes)
    k0, v0 = c.k.clone(), c.v.clone()
    pos = torch.randint(0, c.rope.shape[0], (n_axes, 49), generator=_gen(3), device=DEV, dtype=torch.int32)
    axes = [(7 * i + i // 9) % n_axes for i in range(64)]      # any order
    c.check(c.call(positions=pos, axes=axes), k0, v0, positions=pos, axes=axes)
    if n_axes == 1:
        c.check(c.call(positions=pos[0]), k0, v0, positions=pos)


def test_rows_far_positions_and_sizes_of_values(cuda_lib):
    # a position past 10^6, values of 1e-12 (eps decides) and 1e15
    for scale in (1e-12, 1e15):
        c = Case([3], [3], 4, 2, 16, torch.float32, seed=1, scale=scale)
        c.rope = api.rope_table(1_100_000, D, 1e6, DEV)
        k0, v0 = c.k.clone(), c.v.clone()
        pos = _ints([[0, 999_999, 1_099_999]])
        c.check(c.call(positions=pos), k0, v0, positions=pos)


def test_rows_zeros_and_eps_zero(cuda_lib):
    c = Case([2], [2], 4, 2, 16, torch.float32)
    c.x[0] = 0
    k0, v0 = c.k.clone(), c.v.clone()
    c.check(c.call(), k0, v0)
    c.check(c.call(eps=0.0), k0, v0, eps=0.0, pick=[1])
    assert bool(c.call(eps=0.0)[0].isnan().all())      # 0 / 0


def test_rows_nan_stays_in_its_head(cuda_lib):
    c = Case([3], [20], 4, 2, 16, torch.float32)
    c.x[1, 2 * D + 5] = math.nan
    c.x[2, 5 * D] = math.inf
    q = c.call()
    assert bool(q[1, 2].isnan().all()) and int(q.isnan().any(-1).sum()) == 1
    page, slot = int(c.table[0, 1]), 19 % 16
    assert bool(c.k[page, 1, slot].isnan().any()) and bool(torch.isfinite(c.k[page, 0, slot]).all())


def test_rows_strided_and_outside_every_sequence(cuda_lib):
    c = Case([10, 50], [30, 50], 8, 2, 16, torch.bfloat16)
    wide = torch.full((70, 12 * D + 64), math.nan, dtype=torch.bfloat16, device=DEV)
    wide[4:64, 64:] = c.x
    k0, v0 = c.k.clone(), c.v.clone()
    out = torch.full((70, 8, D), 7.0, device=DEV)
    got = c.call(x=wide[:, 64:], cu=_ints([4, 14, 64]), out=out)
    assert got is out
    c.check(out[4:64], k0, v0)
    assert bool((out[:4] == 7).all()) and bool((out[64:] == 7).all())


POS, PAGE = 2, 1


def _left(c, out, rows):
    assert bool((out[rows] == 7).all()), rows
    rest = [r for r in range(out.shape[0]) if r not in rows]
    assert not bool((out[rest] == 7).any())


def test_rows_left_where_slot_or_position_is_outside(cuda_lib):
    # rows before slot 0, a length past the table, positions past the rotation's table
    c = Case([6, 4, 3], [6, 40, 3], 4, 2, 16, torch.float32)
    new = lambda: torch.full((13, 4, D), 7.0, device=DEV)  # noqa: E731
    out, k0 = new(), c.k.clone()
    c.call(out=out, lens=_ints([4, 49, 3]))
    _left(c, out, [0, 1, 6, 7, 8, 9])
    assert api.check_device_error() == POS
    c.k.copy_(k0)
    pos = _ints([list(range(13)), [5] * 13])
    pos[0, 3], pos[1, 11] = c.rope.shape[0], -1
    out = new()
    c.call(out=out, positions=pos, axes=[0] * 32 + [1] * 32)
    _left(c, out, [3, 11])
    assert api.check_device_error() == POS
    page, slot = int(c.table[0, 0]), 3
    assert torch.equal(c.k[page, :, slot], k0[page, :, slot])      # the whole row is left
    out = new()
    c.call(out=out, cu=_ints([0, 6, 5, 13]))                       # starts that do not ascend
    assert api.check_device_error() == POS
    c.call(out=out, cu=_ints([0, 6, 10, 14]))
    assert api.check_device_error() == POS


def test_rows_whose_page_does_not_exist(cuda_lib):
    c = Case([20, 5], [20, 5], 4, 2, 16, torch.float32)
    good = c.call()
    k0, v0 = c.k.clone(), c.v.clone()
    for bad in (-1, c.k.shape[0]):
        c.table[0, 1] = bad
        assert torch.equal(c.call(), good)
        assert api.check_device_error() == PAGE
        assert torch.equal(c.k, k0) and torch.equal(c.v, v0)       # (written alike before)


def test_rows_most_sequences(cuda_lib):
    r = np.random.default_rng(0)
    rows = [int(n) for n in r.integers(0, 4, 1024)]
    lens = [n + int(m) for n, m in zip(rows, r.integers(0, 40, 1024))]
    c = Case(rows, lens, 4, 2, 16, torch.float32)
    k0, v0 = c.k.clone(), c.v.clone()
    c.check(c.call(), k0, v0)


def test_rows_in_a_graph_and_on_another_stream(cuda_lib):
    c = Case([9, 30], [40, 33], 8, 2, 16, torch.float32)
    cu, lens, out = _ints(c.cu), _ints(c.lens), torch.empty((39, 8, D), device=DEV)
    c.call(cu=cu, lens=lens, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(cu=cu, lens=lens, out=out)
    # other rows and lengths in the same places
    c.x.copy_(torch.randn(c.x.shape, generator=_gen(9), device=DEV))
    c.rows, c.lens, c.cu = [30, 9], [31, 12], [0, 30, 39]
    c.slots = [m - n + j for n, m in zip(c.rows, c.lens) for j in range(n)]
    c.seqs = [b for b, n in enumerate(c.rows) for _ in range(n)]
    cu.copy_(_ints(c.cu))
    lens.copy_(_ints(c.lens))
    k0, v0 = c.k.clone(), c.v.clone()
    graph.replay()
    c.check(out, k0, v0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.call(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, out)


def test_rows_none(cuda_lib):
    c = Case([0], [4], 4, 2, 16, torch.float32)
    assert c.call().shape == (0, 4, D) and api.check_device_error() == 0
