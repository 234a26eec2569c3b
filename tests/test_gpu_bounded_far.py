"""The operators that fill and bound the cache on the GPU where sizes are large or calls overlap: pages past 2^32
elements of the cache, sequences of 150000 tokens, calls on two streams at once."""
import math

import numpy as np
import pytest
import torch

import bounded_reference as ref
from transformer_decode_step_weight_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = 128
SCALE = 1 / math.sqrt(D)
ALL = api.ALL_KEYS
DTYPES = [torch.float32, torch.bfloat16]


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ps", [16, 24])
def test_far_pages_give_what_near_ones_do(cuda_lib, ps, dtype):
    """The same calls on a small cache and on the last pages of one of more than 2^32 elements: every result equal."""
    g = _gen(ps)
    lens, rows, hq, hkv, cu = [700, 90], [130, 40], 8, 2, [0, 130, 170]
    kp, vp, pt = ref.make_cache(g, lens, hkv, ps)
    near = kp.shape[0]
    n_pages = 2 ** 32 // (hkv * ps * D) + near
    far = [torch.empty((n_pages, hkv, ps, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    far[0][n_pages - near:].copy_(kp)
    far[1][n_pages - near:].copy_(vp)
    assert (n_pages - near) * hkv * ps * D >= 2 ** 32 - hkv * ps * D
    qkv = torch.randn((cu[-1], (hq + 2 * hkv) * D), generator=g, device=DEV).to(dtype)
    w = (1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16)
    rope = api.rope_table(800, D, 1e6, DEV)
    start = torch.rand((1, 2, hkv, pt.shape[1] * ps), generator=g, device=DEV)
    got = []
    for k, v, off in ((kp, vp, 0), (*far, n_pages - near)):
        table = torch.where(pt >= 0, pt + off, pt)
        refs = torch.zeros(k.shape[0], dtype=torch.int32, device=DEV)
        refs[table[table >= 0].long()] = 1
        cache = api.PageCache([k], [v], table, _ints(lens), refs)
        sums, n, c = start.clone(), cache.seq_lens, _ints(cu)
        q = api.qk_norm_rope(qkv, w, w, rope, k, v, cache.page_table, c, n, 1e-6)
        out = [q, api.attn_prompt_window(q, k, v, cache.page_table, c, n, SCALE, 200, 4)]
        for last in (0, 7):
            api.attn_key_weights(q, k, cache.page_table, c, n, SCALE, sums[0], last, 300, 4)
        one = api.attn_decode_window(q[:2], k, v, cache.page_table, n, SCALE, 400, 4, key_weights=sums[0])
        out += [one, sums.clone()]
        cache.evict(sums, _ints([333, 50]), 4, 20)
        mine = slice(off, off + near)
        out += [sums, cache.seq_lens, refs[mine], k[mine], v[mine]]
        got.append([t.clone() for t in out])
    assert api.check_device_error() == 0
    for i, (a, b) in enumerate(zip(*got)):
        assert torch.equal(a, b), i


@pytest.mark.parametrize("dtype", DTYPES)
def test_sequences_of_150000_tokens(cuda_lib, dtype):
    g, bf16 = _gen(5), dtype == torch.bfloat16
    lens, hq, hkv, ps = [150000, 131], 4, 2, 16
    rows, cu = [3, 2], [0, 3, 5]
    kp, vp, pt = ref.make_cache(g, lens, hkv, ps)
    q = torch.randn((5, hq, D), generator=g, device=DEV).to(dtype)
    host = [(ref.tokens(kp, pt[b], n), ref.tokens(vp, pt[b], n)) for b, n in enumerate(lens)]
    for window, sinks in ((ALL, 0), (140001, 5)):
        prompt = api.attn_prompt_window(q, kp, vp, pt, _ints(cu), _ints(lens), SCALE, window, sinks).double().cpu()
        sums = torch.zeros((2, hkv, pt.shape[1] * ps), device=DEV)
        api.attn_key_weights(q, kp, pt, _ints(cu), _ints(lens), SCALE, sums, 0, window, sinks)
        total = torch.zeros_like(sums)
        last = q[[2, 4]].contiguous()
        decode = api.attn_decode_window(last, kp, vp, pt, _ints(lens), SCALE, window, sinks, key_weights=total).double().cpu()
        sums, total = sums.double().cpu(), total.double().cpu()
        for b, n in enumerate(lens):
            k, v = host[b]
            all_w, tol_w = torch.zeros((hkv, n), dtype=torch.float64), torch.zeros((hkv, n), dtype=torch.float64)
            for j in range(rows[b]):
                at = n - rows[b] + j
                see = ref.visible(at, n, window, sinks)
                m = int(see.sum())
                want, w, mag, dot = ref.attend(q[cu[b] + j].double().cpu(), k, v, see, SCALE)
                err = (prompt[cu[b] + j] - want).abs() / ref.out_bound(want, mag, dot, m, bf16, 1 if bf16 else 3)
                assert float(err.max()) <= 1, (b, j, float(err.max()))
                all_w += w
                tol_w += w * (ref.weight_bound(dot, m) + 70 * 2.0 ** -24)
            err = (decode[b] - want).abs() / ref.out_bound(want, mag, dot, m, bf16, 2 if bf16 else 3)   # the last row
            assert float(err.max()) <= 1, (b, float(err.max()))
            assert bool(((total[b, :, :n] - w).abs() <= (ref.weight_bound(dot, m) + 2.0 ** -23) * w + 1e-30).all()), b
            assert bool(((sums[b, :, :n] - all_w).abs() <= tol_w + 2.0 ** -23 * all_w + 1e-30).all()), b
            assert not bool(total[b, :, n:].any()) and not bool(sums[b, :, n:].any())
    assert api.check_device_error() == 0


def test_evict_from_150000_tokens(cuda_lib):
    g = _gen(6)
    n, keep, hkv, ps = 150000, 100003, 2, 16
    kp, vp, pt = ref.make_cache(g, [n], hkv, ps)
    old = [ref.tokens(t, pt[0], n) for t in (kp, vp)]
    refs = torch.zeros(kp.shape[0], dtype=torch.int32, device=DEV)
    refs[pt[0].long()] = 1
    table = pt[0].clone()
    cache = api.PageCache([kp], [vp], pt, _ints([n]), refs)
    sums = torch.floor(torch.rand((1, 1, hkv, pt.shape[1] * ps), generator=g, device=DEV) * 1000)   # equal ones among them
    before = sums[0, 0].double().cpu()
    cache.evict(sums, _ints([keep]), 4, 1000)
    assert cache.seq_lens.tolist() == [keep] and int(refs.sum()) == -(-keep // ps)
    for h in range(hkv):
        stay = torch.from_numpy(ref.evict(before[h, :n].numpy(), n, keep, 4, 1000))
        for t, was in zip((kp, vp), old):
            assert torch.equal(ref.tokens(t, table, keep)[:, h], was[stay, h])
        assert torch.equal(sums[0, 0, h, :keep].double().cpu(), before[h, stay]) and not bool(sums[0, 0, h, keep:n].any())
    assert api.check_device_error() == 0


def test_calls_on_two_streams_at_once(cuda_lib):
    """Two of each operator at a time, each with what it allocates itself: the results of calls one after another."""
    g = _gen(7)
    rows, lens, hq, hkv, ps = [90, 200, 32], [900, 200, 1500], 8, 2, 16
    cu = _ints([0, *np.cumsum(rows)])
    n, rope = _ints(lens), api.rope_table(1600, D, 1e6, DEV)
    w = (1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16)
    sides = []
    for dtype in DTYPES:
        kp, vp, pt = ref.make_cache(g, lens, hkv, ps)
        sides.append((torch.randn((sum(rows), (hq + 2 * hkv) * D), generator=g, device=DEV).to(dtype), kp, vp, pt,
                      torch.zeros((3, hkv, pt.shape[1] * ps), device=DEV)))

    def run(side, stream):
        x, kp, vp, pt, zero = side
        with torch.cuda.stream(stream):
            sums, k, v = zero.clone(), kp.clone(), vp.clone()
            q = api.qk_norm_rope(x, w, w, rope, k, v, pt, cu, n, 1e-6)
            out = api.attn_prompt_window(q, k, v, pt, cu, n, SCALE, 150, 4)
            api.attn_key_weights(q, k, pt, cu, n, SCALE, sums, 20)
            api.attn_key_weights(q, k, pt, cu, n, SCALE, sums, 0, 333)
            one = api.attn_decode_window(q[:3], k, v, pt, n, SCALE, 700, 4, key_weights=sums)
            refs = torch.zeros(k.shape[0], dtype=torch.int32, device=DEV)
            refs[torch.where(pt >= 0, pt, 0).long()] = 1
            cache = api.PageCache([k], [v], pt.clone(), n.clone(), refs)
            weighed = sums.clone()
            cache.evict(sums[None], torch.full((3,), 150, dtype=torch.int32, device=DEV), 4, 16)
            return [q, out, one, weighed, sums, k, v, cache.page_table, cache.seq_lens]

    streams = [torch.cuda.Stream() for _ in range(2)]
    want = []
    for side, s in zip(sides, streams):
        torch.cuda.synchronize()
        want.append(run(side, s))
        torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for side, s in zip(sides, streams):
            got.append(run(side, s))
    torch.cuda.synchronize()
    assert api.check_device_error() == 0
    for i, some in enumerate(got):
        for j, (a, b) in enumerate(zip(some, want[i % 2])):
            assert torch.equal(a, b), (i, j)
