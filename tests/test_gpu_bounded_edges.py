"""Calls of the operators that fill and bound the cache at the ends of what they accept: windows and first tokens that
hide nothing, very many sequences, shared pages of which no token goes."""
import math

import numpy as np
import pytest
import torch

import bounded_reference as ref
from test_gpu_evict import CACHE, State
from test_gpu_window import ALL, D, DEV, DTYPES, SCALE, _check_decode, _check_prompt, _check_weights, _gen, _ints, _pack, _pick, _q
from transformer_decode_step_weight_gb300 import api

pytestmark = pytest.mark.gpu
HEAD = 16384     # what of a workspace has to be zero before its first use, at most


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("window,sinks", [(None, ALL), (2 ** 30, 2 ** 30 - 15), (2 ** 30 - 1, 2 ** 30), (None, 2 ** 30 - 16),
                                          (1, ALL)])
def test_neither_window_nor_first_tokens_hide_anything(cuda_lib, window, sinks, dtype):
    # rows of several row tiles (of 32 and 128 tokens), from an empty cache and just behind its first tokens
    for hq, hkv, rows, lens in ((8, 2, [300, 77], [300, 80]), (2, 2, [900, 130], [900, 144])):
        g = _gen(hq)
        kp, vp, pt = ref.make_cache(g, lens, hkv, 16)
        cu, seqs, at = _pack(rows, lens)
        q = _q(g, cu[-1], hq, dtype)
        ws = torch.zeros(api.attn_prompt_workspace_bytes(), dtype=torch.uint8, device=DEV)
        args = (q, kp, vp, pt, _ints(cu), _ints(lens), SCALE)
        out = torch.full((cu[-1], hq, D), math.nan, dtype=dtype, device=DEV)
        api.attn_prompt_window(*args, window, sinks, out=out, workspace=ws)
        _check_prompt(out, q, kp, vp, pt, lens, seqs, at, ALL, 0, rows=_pick(cu[-1], np.random.default_rng(1)))
        assert torch.equal(out, api.attn_prompt_window(*args, workspace=ws))      # the same tiles in the same order
        assert bool((ws[:8192] == 0).all())
        sums = torch.zeros((2, hkv, pt.shape[1] * 16), device=DEV)
        before = sums.clone()
        api.attn_key_weights(q, kp, pt, _ints(cu), _ints(lens), SCALE, sums, window=window, n_sinks=sinks)
        _check_weights(sums, before, q, kp, pt, rows, lens, cu, 0, ALL, 0)
        last, sums = q[[cu[1] - 1, cu[2] - 1]].contiguous(), before.clone()
        one = api.attn_decode_window(last, kp, vp, pt, _ints(lens), SCALE, window, sinks, key_weights=sums)
        _check_decode(one, last, kp, vp, pt, lens, ALL, 0, sums=sums, before=before)
    assert api.check_device_error() == 0


def test_evict_to_first_tokens_on_a_shared_page(cuda_lib):
    # nothing moves where a sequence keeps first tokens alone: a page that it shares is not written
    s = State([90, 0, 100], 2, 2, 16)
    s.cache.fork(_ints([0]), _ints([1]))
    for keep, sinks, lens in (([40, -1, -1], 64, [40, 90, 100]), ([-1, 5, 30], 40, [40, 5, 30]), ([7, 0, 3], 7, [7, 0, 3])):
        s.save()
        s.cache.evict(s.w, _ints(keep), sinks, 3)
        s.check(keep, sinks, 3)
        assert api.check_device_error() == 0 and s.cache.seq_lens.tolist() == lens
    # ... but where others stay, the page that they would move into has to be the sequence's own
    s = State([90, 0], 2, 2, 16)
    s.cache.fork(_ints([0]), _ints([1]))
    s.save()
    s.cache.evict(s.w, _ints([41, -1]), 40, 3)
    assert api.check_device_error() == CACHE and s.same()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [33, 577, 600, 1024])
def test_many_sequences(cuda_lib, n, dtype):
    # more than a warp's look takes (32), than a thread has one of (576), the most; empty ones at both ends and in runs
    g, r = _gen(n), np.random.default_rng(n)
    lens = [int(x) for x in r.integers(0, 90, n)]
    rows = [int(r.integers(0, m + 1)) for m in lens]
    for i in [0, 1, n - 1, *range(n // 3, n // 3 + 20), *r.integers(0, n, n // 8)]:
        rows[i] = 0
    rows[n // 2], lens[n // 2] = 150, 400                  # several row tiles
    hq, hkv, window, sinks = 8, 2, 50, 3
    kp, vp, pt = ref.make_cache(g, lens, hkv, 16)
    cu, seqs, at = _pack(rows, lens)
    q = _q(g, cu[-1], hq, dtype)
    some = set(r.choice(n, 25, replace=False).tolist()) | {0, 2, n // 2, n - 2, n - 1}
    for last, win in ((0, ALL), (0, window), (20, ALL), (20, window)):       # (20 rows of 4 heads: one row tile each)
        before = torch.rand((n, hkv, pt.shape[1] * 16), generator=g, device=DEV) * 0.1
        sums = before.clone()
        api.attn_key_weights(q, kp, pt, _ints(cu), _ints(lens), SCALE, sums, last=last, window=win, n_sinks=sinks)
        _check_weights(sums, before, q, kp, pt, rows, lens, cu, last, win, sinks, seqs=some)
        # each row's weights are 1 together, and what lies behind a sequence stays
        used = torch.tensor([min(x, last) if last else x for x in rows], dtype=torch.float64) * (hq // hkv)
        more = (sums.double() - before.double()).cpu()
        total = more.sum(-1)
        assert bool(((total - used[:, None]).abs() <= 2.0 ** -14 * used[:, None] + 400 * 2.0 ** -23).all())
        behind = torch.arange(more.shape[2])[None] >= torch.tensor(lens)[:, None]
        assert bool((more.transpose(1, 2)[behind] == 0).all()) and bool((more[used == 0] == 0).all())
    out = api.attn_prompt_window(q, kp, vp, pt, _ints(cu), _ints(lens), SCALE, window, sinks)
    _check_prompt(out, q, kp, vp, pt, lens, seqs, at, window, sinks, rows=[i for i, b in enumerate(seqs) if b in some])
    assert api.check_device_error() == 0


@pytest.mark.parametrize("last", [0, 30])
def test_weights_of_a_bf16_q_in_its_own_workspace(cuda_lib, last):
    g = _gen(31)
    rows, lens, hq, hkv = [700, 0, 200], [700, 5, 900], 8, 2
    kp, vp, pt = ref.make_cache(g, lens, hkv, 16)
    cu, _, _ = _pack(rows, lens)
    q = _q(g, cu[-1], hq, torch.bfloat16)
    got = []
    for dtype in (torch.float32, torch.bfloat16, None):
        sums = torch.zeros((3, hkv, pt.shape[1] * 16), device=DEV)
        ws = None
        if dtype is not None:     # with bytes behind it that have to stay
            n = api.attn_key_weights_workspace_bytes(3, cu[-1], hq, hkv, last, dtype)
            room = torch.full((n + 4096,), 255, dtype=torch.uint8, device=DEV)
            room[:HEAD] = 0
            ws = room[:n]
        # (bytes asked for: the allocator does not split a block where less than 1 MB would be left)
        torch.cuda.reset_peak_memory_stats()
        start = torch.cuda.memory_stats()["requested_bytes.all.current"]
        api.attn_key_weights(q, kp, pt, _ints(cu), _ints(lens), SCALE, sums, last=last, workspace=ws)
        used = torch.cuda.memory_stats()["requested_bytes.all.peak"] - start
        assert ws is None or bool((room[n:] == 255).all())
        got.append(sums)
    assert used <= n + 8192 and torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    _check_weights(got[0], torch.zeros_like(got[0]), q, kp, pt, rows, lens, cu, last, ALL, 0)
    assert api.check_device_error() == 0
