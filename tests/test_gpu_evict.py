"""Eviction from the cache by weights on the GPU against a plain implementation, and a run of the operators that fill
and bound the cache together."""
import math

import numpy as np
import pytest
import torch

import bounded_reference as ref
from transformer_decode_step_weight_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = 128
POS, PAGE, CACHE = 2, 1, 32


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class State:
    """A cache whose sequences have these lengths, with random weights, and its copy on the host."""

    def __init__(self, lens, layers, hkv, ps, seed=0, d=D, ties=True, room=0):
        g = _gen(seed)
        _, _, table = ref.make_cache(g, lens, 1, ps, room=room)
        self.ps, n_pages = ps, int(table.max()) + 4
        shape = (n_pages, hkv, ps, d)
        self.k = [torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16) for _ in range(layers)]
        self.v = [torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16) for _ in range(layers)]
        refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
        refs[table[table >= 0].long()] = 1
        self.cache = api.PageCache(self.k, self.v, table, _ints(lens), refs)
        self.w = torch.rand((layers, len(lens), hkv, table.shape[1] * ps), generator=g, device=DEV)
        if ties:    # few values, so that the border falls among equal ones
            self.w = torch.floor(self.w * 6) / 6
        self.save()

    def save(self):
        c = self.cache
        self.old = [t.clone().cpu() for t in (c.page_table, c.seq_lens, c.refs, self.w, *self.k, *self.v)]

    def same(self):
        c = self.cache
        return all(torch.equal(a.cpu().nan_to_num(7), b.nan_to_num(7))
                   for a, b in zip((c.page_table, c.seq_lens, c.refs, self.w, *self.k, *self.v), self.old))

    def check(self, keep, sinks, recent):
        table, lens, refs, w, *kv = self.old
        L, ps = len(self.k), self.ps
        want_w, want = w.clone(), [t.clone() for t in kv]
        for b, n in enumerate(lens.tolist()):
            m = n if keep[b] < 0 or keep[b] >= n else keep[b]
            if m == n:
                continue
            at = torch.arange(n)
            page, slot = table[b].long()[at // ps], at % ps
            for l in range(L):
                for h in range(w.shape[2]):
                    stay = torch.from_numpy(ref.evict(w[l, b, h, :n].double().numpy(), n, keep[b], sinks, recent))
                    want_w[l, b, h, :m] = w[l, b, h, stay]
                    want_w[l, b, h, m:n] = 0
                    for t, old in ((want[l], kv[l]), (want[L + l], kv[L + l])):
                        t[page[:m], h, slot[:m]] = old[page[stay], h, slot[stay]]
            for i in range(-(-m // ps), -(-n // ps)):
                refs[table[b, i]] -= 1
                table[b, i] = -1
            lens[b] = m
        c = self.cache
        assert torch.equal(c.page_table.cpu(), table) and torch.equal(c.seq_lens.cpu(), lens)
        assert torch.equal(c.refs.cpu(), refs)
        assert torch.equal(self.w.cpu().nan_to_num(7), want_w.nan_to_num(7))
        for i, (got, t) in enumerate(zip([*self.k, *self.v], want)):
            assert torch.equal(got.cpu(), t), i


CASES = [   # lengths, layers, kv heads, page size, budgets, first tokens, last tokens
    ([40], 1, 1, 16, [10], 0, 0),
    ([40], 1, 2, 16, [39], 2, 3),
    ([40, 7, 100], 2, 2, 16, [12, 7, 64], 4, 8),
    ([40, 7, 100], 2, 2, 16, [-1, 3, 200], 4, 8),
    ([1, 2, 0, 3], 1, 1, 1, [0, 1, 0, 2], 1, 1),
    ([300, 5], 3, 2, 7, [123, 4], 5, 50),
    ([300, 33], 1, 4, 24, [10, 30], 100, 100),       # fewer than the first ones
    ([300, 33], 1, 4, 24, [110, 20], 100, 100),      # ... than the first and last together
    ([2500], 2, 1, 16, [1300], 4, 256),
    ([1700, 900], 1, 2, 64, [1699, 1], 0, 0),
    ([5000], 1, 1, 128, [4097], 7, 1030),
    ([600] * 5, 1, 2, 16, [100, 200, 300, 400, 500], 3, 2),
]


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("lens,layers,hkv,ps,keep,sinks,recent", CASES)
def test_evict(cuda_lib, lens, layers, hkv, ps, keep, sinks, recent, ties):
    s = State(lens, layers, hkv, ps, seed=sum(lens), ties=ties)
    s.cache.evict(s.w, _ints(keep), sinks, recent)
    s.check(keep, sinks, recent)
    assert api.check_device_error() == 0


@pytest.mark.parametrize("seed", range(8))
def test_evict_ragged_and_again(cuda_lib, seed):
    r = np.random.default_rng(seed)
    B = int(r.integers(1, 12)) if seed < 6 else 40
    lens = [int(x) for x in 2 ** r.uniform(0, 11.5, B)]
    s = State(lens, int(r.integers(1, 4)) if seed < 6 else 9, int(r.choice([1, 2, 8])) if seed < 6 else 2, int(r.choice([1, 7, 16, 24, 128])), seed=seed, ties=seed % 2 == 0)
    for _ in range(3):
        lens = s.cache.seq_lens.tolist()
        keep = [int(r.integers(-1, n + 2)) for n in lens]
        sinks, recent = int(r.integers(0, 20)), int(r.integers(0, 60))
        s.save()
        s.cache.evict(s.w, _ints(keep), sinks, recent)
        s.check(keep, sinks, recent)
    assert api.check_device_error() == 0


@pytest.mark.parametrize("what", ["zeros", "alike", "rising", "falling", "signs", "odd"])
def test_evict_weights_of_every_kind(cuda_lib, what):
    s = State([700, 90], 2, 2, 16)
    w = s.w
    if what == "zeros":
        w.zero_()
    elif what == "alike":
        w.fill_(0.25)
    elif what in ("rising", "falling"):
        i = torch.arange(w.shape[-1], device=DEV, dtype=torch.float32)
        w.copy_((i if what == "rising" else 1000 - i).expand_as(w))
    elif what == "signs":      # below zero, both zeros (equal), numbers below the normal range
        w.sub_(0.5)
        w[..., ::3] = 0.0
        w[..., 1::3] = -0.0
        w[..., 2::12] = 1e-42
    else:
        w[..., ::5] = math.nan
        w[..., 1::5] = math.inf
        w[..., 2::5] = -math.inf
    s.save()
    s.cache.evict(s.w, _ints([300, 40]), 4, 30)
    s.check([300, 40], 4, 30)
    assert api.check_device_error() == 0


@pytest.mark.parametrize("d,layers", [(8, 1), (64, 70), (256, 2)])
def test_evict_head_sizes_and_many_layers(cuda_lib, d, layers):
    s = State([130, 60], layers, 2, 16, d=d)
    s.cache.evict(s.w, _ints([70, 31]), 2, 9)
    s.check([70, 31], 2, 9)
    assert api.check_device_error() == 0


@pytest.mark.parametrize("n", [500, 1300])
def test_evict_many_sequences(cuda_lib, n):
    r = np.random.default_rng(5)
    lens = [int(x) for x in r.integers(0, 60, n)]
    keep = [int(x) for x in r.integers(-1, 60, n)]
    lens[7], keep[7] = 2500, 1203
    s = State(lens, 1, 1, 16)
    s.cache.evict(s.w, _ints(keep), 2, 5)
    s.check(keep, 2, 5)
    assert api.check_device_error() == 0


def test_evict_changes_nothing_where_it_cannot_be_whole(cuda_lib):
    # sequence 1 shares its pages with 2: the pages that would be written are shared
    s = State([100, 90, 0], 2, 2, 16)
    c = s.cache
    c.fork(_ints([1]), _ints([2]))
    s.save()
    c.evict(s.w, _ints([50, 40, -1]), 4, 8)
    assert api.check_device_error() == CACHE and s.same()
    c.evict(s.w, _ints([50, 40, 40]), 4, 8)
    assert api.check_device_error() == CACHE and s.same()
    # shared first pages that stay as they are, and shared ones behind the new length, are no hindrance
    c.trim(_ints([-1, -1, 32]))
    s.save()
    c.evict(s.w, _ints([50, 80, -1]), 32, 8)
    s.check([50, 80, -1], 32, 8)
    assert api.check_device_error() == 0
    s = State([100, 90], 1, 1, 16)
    for entry in (-1, 10 ** 6):
        s.cache.page_table[0, 3] = entry
        s.save()
        s.cache.evict(s.w, _ints([50, 40]), 4, 8)
        assert api.check_device_error() == CACHE | PAGE and s.same()
    s.cache.seq_lens[0] = s.cache.page_table.shape[1] * 16 + 1
    s.save()
    s.cache.evict(s.w, _ints([50, 40]), 4, 8)
    assert api.check_device_error() & CACHE and s.same()
    s.cache.evict(s.w, _ints([-1, 40]), 4, 8)           # the broken sequence left out
    s.check([-1, 40], 4, 8)
    assert api.check_device_error() == 0


def test_evict_in_a_graph_and_on_another_stream(cuda_lib):
    s = State([800, 300], 2, 2, 16)
    c, keep = s.cache, _ints([800, 300])
    c.evict(s.w, keep, 4, 16)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.evict(s.w, keep, 4, 16)
    for k in ([500, 300], [333, 7], [333, 7], [0, 6]):
        s.save()
        keep.copy_(_ints(k))
        graph.replay()
        s.check(k, 4, 16)
    s = State([800, 300], 2, 2, 16, seed=3)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    keep = _ints([400, 200])
    other.wait_stream(torch.cuda.current_stream())
    s.cache.evict(s.w, keep, 4, 16, stream=other)
    torch.cuda.current_stream().wait_stream(other)
    s.check([400, 200], 4, 16)
    assert api.check_device_error() == 0
    with pytest.raises(ValueError, match="key_weights"):
        s.cache.evict(s.w[:1], keep)
    with pytest.raises(api.QDError, match="n_sinks"):
        s.cache.evict(s.w, keep, -1)


def test_prompts_and_tokens_through_a_bounded_cache(cuda_lib):
    """Two prompts and then tokens, the cache cut to a budget every few tokens: each row's attention is that of a
    host's own list of (K, V), kept by its own sums of weights."""
    g, r = _gen(21), np.random.default_rng(21)
    layers, hq, hkv, ps, budget, sinks, recent, last = 2, 8, 2, 16, 96, 4, 24, 16
    B, width, n_pages = 2, 20, 50
    shape = (n_pages, hkv, ps, D)
    kc = [torch.zeros(shape, dtype=torch.bfloat16, device=DEV) for _ in range(layers)]
    vc = [torch.zeros(shape, dtype=torch.bfloat16, device=DEV) for _ in range(layers)]
    cache = api.PageCache.empty(kc, vc, B, width)
    sums = torch.zeros((layers, B, hkv, width * ps), device=DEV)
    rope = api.rope_table(600, D, 1e6, DEV)
    qn, kn = ((1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16) for _ in range(2))
    scale = 1 / math.sqrt(D)
    host = [[[[], [], []] for _ in range(B)] for _ in range(layers)]      # K, V and weights per kv head

    def rows_of(n):
        return torch.randn((n, (hq + 2 * hkv) * D), generator=g, device=DEV) * 1.5

    def mirror(l, b, pos, x):
        cs = rope[pos].double().cpu()
        h = x.double().cpu().view(-1, D)
        k, _, _ = ref.norm_rope(h[hq:hq + hkv], kn.double().cpu(), cs, 1e-6, False)
        q, _, _ = ref.norm_rope(h[:hq], qn.double().cpu(), cs, 1e-6, False)
        kk, vv, ww = host[l][b]
        kk.append(k.to(torch.bfloat16).double())
        vv.append(h[hq + hkv:].to(torch.bfloat16).double())
        ww.append(torch.zeros(hkv, dtype=torch.float64))
        return q

    def attend(l, b, q, count):
        kk, vv, ww = (torch.stack(t) for t in host[l][b])
        out, w, _, _ = ref.attend(q, kk, vv, torch.ones(len(kk), dtype=torch.bool), scale)
        if count:
            host[l][b][2] = list(ww + w.T)
        return out

    # K in the cache is rounded to bf16 after a sum in f32: one of its roundings may go the other way (2^-8 of a value
    # of some 2, in a dot of 128 of them with weights near 1/100): the comparison's limit
    near = 2.0 ** -6
    prompt = [150, 61]
    cache.extend(_ints(prompt))
    cu, pos = _ints([0, *np.cumsum(prompt)]), [int(n) for n in prompt]
    for l in range(layers):
        x = rows_of(sum(prompt))
        q = api.qk_norm_rope(x, qn, kn, rope, kc[l], vc[l], cache.page_table, cu, cache.seq_lens, 1e-6)
        out = api.attn_prompt_window(q, kc[l], vc[l], cache.page_table, cu, cache.seq_lens, scale)
        api.attn_key_weights(q, kc[l], cache.page_table, cu, cache.seq_lens, scale, sums[l], last=last)
        at = 0
        for b, n in enumerate(prompt):
            for j in range(n):
                want = attend(l, b, mirror(l, b, j, x[at]), j >= n - last)
                assert float((out[at].double().cpu() - want).abs().max()) < near, (l, b, j)
                at += 1
    one, cu1 = _ints([1, 1]), _ints([0, 1, 2])
    for step in range(40):
        if step % 13 == 0:
            keep = [min(budget, len(host[0][b][0])) for b in range(B)]
            # the device's sums choose for both sides where two of them are close: they are compared first
            for l in range(layers):
                for b in range(B):
                    ww = torch.stack(host[l][b][2]).T
                    got = sums[l, b, :, :ww.shape[1]].double().cpu()
                    assert float((got - ww).abs().max()) < near
                    for h in range(hkv):
                        stay = ref.evict(got[h].numpy(), ww.shape[1], keep[b], sinks, recent)
                        for t in host[l][b]:
                            col = [t[i][h].clone() for i in stay]
                            for i, c in enumerate(col):
                                t[i] = t[i].clone()
                                t[i][h] = c
                    host[l][b] = [t[:keep[b]] for t in host[l][b]]
            cache.evict(sums, _ints(keep), sinks, recent)
            assert cache.seq_lens.tolist() == keep
        cache.extend(one)
        where = _ints([[p for p in pos]])
        for l in range(layers):
            x = rows_of(B)
            q = api.qk_norm_rope(x, qn, kn, rope, kc[l], vc[l], cache.page_table, cu1, cache.seq_lens, 1e-6, positions=where)
            out = api.attn_decode_window(q, kc[l], vc[l], cache.page_table, cache.seq_lens, scale, key_weights=sums[l])
            for b in range(B):
                want = attend(l, b, mirror(l, b, pos[b], x[b]), True)
                assert float((out[b].double().cpu() - want).abs().max()) < near, (step, l, b)
        pos = [p + 1 for p in pos]
    assert api.check_device_error() == 0 and int((cache.refs > 0).sum()) <= 2 * -(-(budget + 14) // ps)
