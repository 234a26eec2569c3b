"""The serving operators on the GPU against plain 64-bit implementations: attention of packed
prompts and of sequences that share a prefix, page operations, sampled verification, and a run
of them together."""
import math

import numpy as np
import pytest
import torch

import serving_reference as ref
from transformer_decode_step_weight_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = 128
SCALE = 1 / math.sqrt(D)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cache(g, lens, hkv, ps, shared=None, spare=3):
    """Caches and page table of sequences of these lengths; `shared`: per sequence (group, whole pages shared)."""
    rows, used, heads = [], 0, {}
    for b, n in enumerate(lens):
        row = []
        if shared is not None:
            grp, pages = shared[b]
            if grp not in heads:
                heads[grp] = list(range(used, used + pages))
                used += pages
            row = list(heads[grp])
        need = max(0, -(-n // ps) - len(row))
        rows.append(row + list(range(used, used + need)))
        used += need
    n_pages = used + spare
    perm = torch.randperm(n_pages, generator=g, device=DEV).tolist()
    width = max(1, max(len(r) for r in rows))
    pt = _ints([[perm[p] for p in r] + [-1] * (width - len(r)) for r in rows])
    kp = torch.randn((n_pages, hkv, ps, D), generator=g, device=DEV).to(torch.bfloat16)
    vp = torch.randn((n_pages, hkv, ps, D), generator=g, device=DEV).to(torch.bfloat16)
    return kp, vp, pt


def _check_rows(got, q, kp, vp, pt, seqs, seen, rows=None, scale=SCALE):
    """Rows of `got` against the 64-bit form: row r belongs to sequence seqs[r] and sees seen[r] keys."""
    bf16 = q.dtype == torch.bfloat16
    got, q = got.double().cpu(), q.double().cpu()
    kv = {}
    for r in range(len(seqs)) if rows is None else rows:
        b, n = seqs[r], max(0, seen[r])
        if b not in kv:
            m = max(0, max(s for x, s in zip(seqs, seen) if x == b))
            kv[b] = ref.gather(kp, pt[b], m), ref.gather(vp, pt[b], m)
        out, mag, vmax, dot = ref.attend(q[r], *kv[b], n, scale)
        tol = ref.attention_bound(out, mag, vmax, dot, n, bf16)
        err = (got[r] - out).abs()
        assert bool((err <= tol).all()), (r, b, n, float((err / tol).max()), float(err.max()))


def _pack(rows, lens):
    cu = [0]
    for n in rows:
        cu.append(cu[-1] + n)
    seqs = [b for b, n in enumerate(rows) for _ in range(n)]
    seen = [m - n + j + 1 for n, m in zip(rows, lens) for j in range(n)]
    return cu, seqs, seen


PROMPTS = [
    ([1], [1], 4, 2, 16),
    ([1, 1, 1], [1, 17, 300], 8, 8, 16),
    ([5], [5], 8, 1, 16),
    ([128], [128], 4, 4, 16),
    ([129, 0, 127], [129, 40, 127], 4, 2, 32),
    ([64, 65, 3, 31], [64, 65, 1000, 331], 32, 8, 16),
    ([300, 17], [300, 900], 16, 2, 64),
    ([33, 70], [129, 70], 4, 2, 7),
    ([40, 200], [40, 1500], 8, 2, 24),
    ([16, 20], [5, 20], 4, 2, 16),          # rows before position 0 see nothing
    ([9, 4], [0, 0], 4, 1, 16),             # sequences without any key
    ([1], [5000], 8, 1, 128),               # one row, a long cache: split over the SMs
    ([600], [2100], 8, 2, 256),
    ([2, 0, 0, 1], [2, 0, 7, 257], 2, 2, 1),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,lens,hq,hkv,ps", PROMPTS)
def test_prompt_attention(cuda_lib, rows, lens, hq, hkv, ps, dtype):
    g = _gen(sum(rows) + hq)
    kp, vp, pt = _cache(g, lens, hkv, ps)
    cu, seqs, seen = _pack(rows, lens)
    q = torch.randn((cu[-1], hq, D), generator=g, device=DEV).to(dtype)
    ws = torch.zeros(api.attn_prompt_workspace_bytes(), dtype=torch.uint8, device=DEV)
    first = api.attn_prompt(q, kp, vp, pt, _ints(cu), _ints(lens), SCALE, workspace=ws)
    again = api.attn_prompt(q, kp, vp, pt, _ints(cu), _ints(lens), SCALE, workspace=ws)
    assert torch.equal(first, again)   # the workspace is left ready, and the order of sums fixed
    pick = sorted(set(list(range(min(40, cu[-1]))) + list(range(0, cu[-1], 13)) + list(range(max(0, cu[-1] - 20), cu[-1]))))
    _check_rows(first, q, kp, vp, pt, seqs, seen, pick)
    assert api.check_device_error() == 0


@pytest.mark.parametrize("seed,hq,hkv,ps,n", [(0, 8, 1, 24, 60), (1, 4, 4, 7, 60), (2, 32, 8, 16, 16), (3, 16, 2, 64, 7),
                                              (4, 8, 8, 16, 40), (5, 8, 2, 128, 3), (6, 8, 4, 32, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompt_attention_ragged_batches_again_and_again(cuda_lib, seed, hq, hkv, ps, n, dtype):
    # row tiles of every length one after another in a CTA, whole and in pieces; the same bits each time
    g, r = _gen(60 + seed), np.random.default_rng(seed)
    lens = [int(x) for x in 2 ** r.uniform(0, 12.5, n)]
    rows = [min(m, int(x)) for m, x in zip(lens, 2 ** r.uniform(0, 11, n))]
    kp, vp, pt = _cache(g, lens, hkv, ps)
    cu, seqs, seen = _pack(rows, lens)
    q = (torch.randn((cu[-1], hq, D), generator=g, device=DEV) * (10 if seed % 3 == 0 else 1)).to(dtype)
    args = (q, kp, vp, pt, _ints(cu), _ints(lens), SCALE)
    ws = torch.zeros(api.attn_prompt_workspace_bytes(), dtype=torch.uint8, device=DEV)
    first = api.attn_prompt(*args, workspace=ws)
    for _ in range(12):
        assert torch.equal(first, api.attn_prompt(*args, workspace=ws))
    pick = sorted(r.choice(cu[-1], min(60, cu[-1]), replace=False).tolist())
    _check_rows(first, q, kp, vp, pt, seqs, seen, pick)
    assert api.check_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompt_attention_leaves_other_rows_and_takes_strided_q(cuda_lib, dtype):
    g = _gen(5)
    rows, lens, hq, hkv = [10, 50], [30, 50], 8, 2
    kp, vp, pt = _cache(g, lens, hkv, 16)
    qkv = torch.randn((70, hq + 2 * hkv, D), generator=g, device=DEV).to(dtype)
    qkv[:4] = math.nan      # rows outside every sequence are not read
    qkv[64:] = math.nan
    out = torch.full((70, hq, D), 7.0, dtype=dtype, device=DEV)
    cu, seqs, seen = _pack(rows, lens)
    api.attn_prompt(qkv[:, :hq], kp, vp, pt, _ints([c + 4 for c in cu]), _ints(lens), SCALE, out=out)
    _check_rows(out[4:64], qkv[4:64, :hq], kp, vp, pt, seqs, seen)
    assert bool((out[:4] == 7).all()) and bool((out[64:] == 7).all())
    assert api.check_device_error() == 0


@pytest.mark.parametrize("ps", [16, 64, 24])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompt_attention_unseen_values(cuda_lib, ps, bad, dtype):
    # NaN and infinities behind a sequence's last token, and in tokens that come after a row
    g = _gen(6)
    rows, lens, hq, hkv = [90, 20], [150, 45], 8, 2
    kp, vp, pt = _cache(g, lens, hkv, ps)
    cu, seqs, seen = _pack(rows, lens)
    q = torch.randn((cu[-1], hq, D), generator=g, device=DEV).to(dtype)
    for b, n in enumerate(lens):
        if n % ps:
            for t in (kp, vp):
                t[int(pt[b, n // ps]), :, n % ps:] = bad
    # token 100 of sequence 0 is poisoned: only its rows from position 100 on may see it
    for t in (kp, vp):
        t[int(pt[0, 100 // ps]), 0, 100 % ps, 5] = bad
        t[int(pt[0, 100 // ps]), 1, 100 % ps] = bad
    out = api.attn_prompt(q, kp, vp, pt, _ints(cu), _ints(lens), SCALE)
    ok = [r for r in range(cu[-1]) if seqs[r] == 1 or seen[r] <= 100]
    clean_k, clean_v = kp.clone(), vp.clone()
    for t in (clean_k, clean_v):
        t[~torch.isfinite(t)] = 0
    _check_rows(out, q, clean_k, clean_v, pt, seqs, seen, ok)
    assert bool(torch.isfinite(out[ok]).all())
    late = [r for r in range(cu[-1]) if seqs[r] == 0 and seen[r] > 100]
    if math.isnan(bad):
        assert bool(torch.isnan(out[late][:, :, 5]).all())      # and they do see it


def test_prompt_attention_value_only_infinity_reaches_the_rows_that_see_it(cuda_lib):
    g = _gen(7)
    rows, lens, hq, hkv = [140], [200], 4, 2
    kp, vp, pt = _cache(g, lens, hkv, 16)
    cu, seqs, seen = _pack(rows, lens)
    q = torch.randn((cu[-1], hq, D), generator=g, device=DEV)
    vp[int(pt[0, 170 // 16]), :, 170 % 16, 3] = math.inf
    vp[int(pt[0, 180 // 16]), :, 180 % 16, 9] = -math.inf
    out = api.attn_prompt(q, kp, vp, pt, _ints(cu), _ints(lens), SCALE)
    at = torch.tensor(seen, device=DEV)
    assert bool((torch.isposinf(out[:, :, 3]) == (at > 170)[:, None]).all())
    assert bool((torch.isneginf(out[:, :, 9]) == (at > 180)[:, None]).all())
    rest = [d for d in range(D) if d not in (3, 9)]
    assert bool(torch.isfinite(out[:, :, rest]).all())


def test_prompt_attention_large_scores(cuda_lib):
    # scores of several hundred: the running maximum moves by far more than an exponent's range
    g = _gen(8)
    rows, lens, hq, hkv = [200], [700], 4, 2
    kp, vp, pt = _cache(g, lens, hkv, 16)
    cu, seqs, seen = _pack(rows, lens)
    q = (torch.randn((cu[-1], hq, D), generator=g, device=DEV) * 40).to(torch.bfloat16)
    out = api.attn_prompt(q, kp, vp, pt, _ints(cu), _ints(lens), SCALE)
    _check_rows(out, q, kp, vp, pt, seqs, seen, range(0, 200, 7))


def test_prompt_attention_far_pages(cuda_lib):
    # pages whose byte and element offsets pass 32 bits
    g = _gen(9)
    hq, hkv, ps, n_pages, n = 8, 8, 16, 140000, 300
    kp = torch.empty((n_pages, hkv, ps, D), dtype=torch.bfloat16, device=DEV)
    vp = torch.empty_like(kp)
    ids = list(range(n_pages - 1, n_pages - 1 - 19 * 3, -3))
    pt = _ints([ids, ids[::-1]])
    kp[pt.flatten().long()] = torch.randn((38, hkv, ps, D), generator=g, device=DEV).to(torch.bfloat16)
    vp[pt.flatten().long()] = torch.randn((38, hkv, ps, D), generator=g, device=DEV).to(torch.bfloat16)
    rows, lens = [40, 1], [n, n]
    cu, seqs, seen = _pack(rows, lens)
    q = torch.randn((cu[-1], hq, D), generator=g, device=DEV)
    out = api.attn_prompt(q, kp, vp, pt, _ints(cu), _ints(lens), SCALE)
    _check_rows(out, q, kp, vp, pt, seqs, seen)
    out = api.attn_decode_shared(q[:2].contiguous(), kp, vp, pt, _ints(lens), _ints([0, 2]), _ints([0]), SCALE)
    _check_rows(out, q[:2], kp, vp, pt, [0, 1], lens)
    assert api.check_device_error() == 0


def test_prompt_attention_device_errors(cuda_lib):
    g = _gen(10)
    hq, hkv, ps = 4, 2, 16
    kp, vp, pt = _cache(g, [64, 64], hkv, ps)
    q = torch.randn((20, hq, D), generator=g, device=DEV)
    out = torch.full((20, hq, D), 3.0, device=DEV)
    for cu in ([0, 15, 10], [0, 10, 21], [-1, 5, 20]):   # not ascending, past n_rows, below 0
        api.attn_prompt(q, kp, vp, pt, _ints(cu), _ints([64, 64]), SCALE, out=out)
        assert api.check_device_error() == 2
        assert bool((out == 3).all())
    # a length past the table: that sequence is left, the other is right
    api.attn_prompt(q, kp, vp, pt, _ints([0, 10, 20]), _ints([65, 64]), SCALE, out=out)
    assert api.check_device_error() == 2
    assert bool((out[:10] == 3).all())
    _check_rows(out, q, kp, vp, pt, [0] * 10 + [1] * 10, [0] * 10 + list(range(55, 65)), range(10, 20))
    # a page id outside the cache is not followed
    pt[1, 1] = kp.shape[0]
    api.attn_prompt(q, kp, vp, pt, _ints([0, 10, 20]), _ints([64, 64]), SCALE, out=out)
    assert api.check_device_error() == 1
    _check_rows(out, q, kp, vp, pt, [0] * 10 + [1] * 10, list(range(55, 65)) + [0] * 10, range(10))


SHARED = [
    # groups as (members, shared tokens), tails, hq, hkv, page
    ([(1, 40)], [9], 4, 2, 16),
    ([(4, 300)], [0, 1, 40, 17], 16, 8, 16),
    ([(3, 0), (2, 130)], [5, 0, 64, 1, 700], 8, 2, 16),
    ([(40, 1000)], list(range(40)), 32, 8, 16),
    ([(70, 260)], [i % 3 for i in range(70)], 8, 1, 32),
    ([(5, 2000), (1, 50), (7, 129)], [300, 2, 0, 90, 31, 8, 1, 2, 3, 4, 5, 6, 7], 8, 8, 64),
    ([(6, 777)], [1, 2, 3, 4, 5, 6], 4, 2, 7),
    ([(2, 3000)], [1500, 3], 2, 2, 24),
    ([(100, 1500), (3, 700), (20, 300)], [i % 5 for i in range(123)], 8, 1, 16),   # teams of 7 CTAs
    ([(80, 400)], [2] * 80, 8, 2, 64),
    ([(150, 300)], [i % 2 for i in range(150)], 8, 1, 16),   # more row tiles than a team has members
    ([(3, 150)], [1, 0, 3], 4, 1, 1),
]


# QD_SHARED_MIN_MB 0: the prefixes are shared whatever that spares; default: at these sizes they are not
@pytest.mark.parametrize("min_mb", ["0", None])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("groups,tails,hq,hkv,ps", SHARED)
def test_shared_prefix_attention(cuda_lib, monkeypatch, groups, tails, hq, hkv, ps, dtype, min_mb):
    if min_mb is not None:
        monkeypatch.setenv("QD_SHARED_MIN_MB", min_mb)
    g = _gen(len(tails) + hq)
    who = [i for i, (n, _) in enumerate(groups) for _ in range(n)]
    lens = [groups[i][1] + t for i, t in zip(who, tails)]
    shared = [(i, groups[i][1] // ps) for i in who]
    kp, vp, pt = _cache(g, lens, hkv, ps, shared)
    B = len(lens)
    cu = [0]
    for n, _ in groups:
        cu.append(cu[-1] + n)
    q = torch.randn((B, hq, D), generator=g, device=DEV).to(dtype)
    # whole shared pages, and part of one
    ws = torch.zeros(api.attn_shared_workspace_bytes(B, hq, hkv), dtype=torch.uint8, device=DEV)
    for cut in (0, 3):
        sl = [max(0, s // ps * ps - cut) for _, s in groups]
        args = (q, kp, vp, pt, _ints(lens), _ints(cu), _ints(sl), SCALE)
        out = api.attn_decode_shared(*args, workspace=ws)
        assert torch.equal(out, api.attn_decode_shared(*args, workspace=ws))
        _check_rows(out, q, kp, vp, pt, list(range(B)), lens)
    if dtype == torch.float32:
        paged = api.attn_decode_paged(q, kp, vp, pt, _ints(lens), SCALE)
        _check_rows(paged, q, kp, vp, pt, list(range(B)), lens)   # the same operator
    assert api.check_device_error() == 0


@pytest.mark.parametrize("min_mb", ["0", "80"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_shared_prefix_attention_short_empty_and_outside_sequences(cuda_lib, monkeypatch, dtype, min_mb):
    monkeypatch.setenv("QD_SHARED_MIN_MB", min_mb)
    g = _gen(21)
    ps, hq, hkv, shared = 16, 8, 2, 200
    lens = [250, 0, 100, 200, 201, 5, 33]
    kp, vp, pt = _cache(g, [250] * 7, hkv, ps, [(0, 13)] * 7)
    vp[pt[0, 13:].long()] = math.nan       # the first sequence's own pages: nobody else's keys
    q = torch.randn((7, hq, D), generator=g, device=DEV).to(dtype)
    out = torch.full((7, hq, D), 5.0, dtype=dtype, device=DEV)
    # sequence 6 lies behind the last group
    api.attn_decode_shared(q, kp, vp, pt, _ints(lens), _ints([0, 6]), _ints([shared]), SCALE, out=out)
    _check_rows(out, q, kp, vp, pt, list(range(7)), lens, range(1, 6))
    assert bool((out[1] == 0).all()) and bool((out[6] == 5).all())
    assert bool(torch.isnan(out[0]).any())
    assert api.check_device_error() == 0


@pytest.mark.parametrize("min_mb", ["0", "80"])
def test_shared_prefix_attention_device_errors(cuda_lib, monkeypatch, min_mb):
    monkeypatch.setenv("QD_SHARED_MIN_MB", min_mb)
    g = _gen(22)
    kp, vp, pt = _cache(g, [64] * 4, 2, 16, [(0, 2)] * 4)
    q = torch.randn((4, 4, D), generator=g, device=DEV)
    out = torch.full((4, 4, D), 3.0, device=DEV)
    api.attn_decode_shared(q, kp, vp, pt, _ints([64] * 4), _ints([0, 5]), _ints([32]), SCALE, out=out)
    assert api.check_device_error() == 2 and bool((out == 3).all())
    api.attn_decode_shared(q, kp, vp, pt, _ints([64, 65, -1, 64]), _ints([0, 4]), _ints([32]), SCALE, out=out)
    assert api.check_device_error() == 2
    _check_rows(out, q, kp, vp, pt, [0, 1, 2, 3], [64] * 4, [0, 3])
    assert bool((out[1:3] == 3).all())


@pytest.mark.parametrize("op", ["prompt", "shared"])
def test_attention_in_a_graph_and_on_another_stream(cuda_lib, monkeypatch, op):
    monkeypatch.setenv("QD_SHARED_MIN_MB", "0")
    g = _gen(23)
    hq, hkv, ps = 8, 2, 16
    lens = [500, 300, 420]
    kp, vp, pt = _cache(g, lens, hkv, ps, [(0, 15)] * 3)
    q = torch.randn((3, hq, D), generator=g, device=DEV)
    ln, cu, sl = _ints(lens), _ints([0, 1, 2, 3]), _ints([240])

    def call(**kw):
        if op == "prompt":
            return api.attn_prompt(q, kp, vp, pt, cu, ln, SCALE, **kw)
        return api.attn_decode_shared(q, kp, vp, pt, ln, cu[::3].contiguous(), sl, SCALE, **kw)

    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    nbytes = api.attn_prompt_workspace_bytes() if op == "prompt" else api.attn_shared_workspace_bytes(3, hq, hkv)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device=DEV)
    out = torch.zeros_like(want)
    cu3 = cu[::3].contiguous()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        if op == "prompt":
            api.attn_prompt(q, kp, vp, pt, cu, ln, SCALE, out=out, workspace=ws)
        else:
            api.attn_decode_shared(q, kp, vp, pt, ln, cu3, sl, SCALE, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    # the lengths are read on the device: the same graph after the sequences grew shorter
    ln.copy_(_ints([241, 17, 420]))
    graph.replay()
    _check_rows(out, q, kp, vp, pt, [0, 1, 2], [241, 17, 420])
    assert api.check_device_error() == 0


@pytest.mark.parametrize("min_mb", ["0", "80"])
def test_one_workspace_for_calls_of_different_sizes(cuda_lib, monkeypatch, min_mb):
    monkeypatch.setenv("QD_SHARED_MIN_MB", min_mb)
    # split sequences (tickets) of one batch size after another, in one workspace
    g = _gen(24)
    hq, hkv, ps = 8, 2, 16
    ws = torch.zeros(max(api.attn_shared_workspace_bytes(b, hq, hkv) for b in (1, 3, 40)), dtype=torch.uint8,
                     device=DEV)
    for B in (40, 1, 3, 40, 2):
        lens = [700 + 40 * i for i in range(B)]
        lens[0] = 5000
        kp, vp, pt = _cache(g, lens, hkv, ps, [(0, 10)] * B)
        q = torch.randn((B, hq, D), generator=g, device=DEV)
        for _ in range(2):
            out = api.attn_decode_shared(q, kp, vp, pt, _ints(lens), _ints([0, B]), _ints([160]), SCALE, workspace=ws)
        _check_rows(out, q, kp, vp, pt, list(range(B)), lens, sorted({0, B // 2, B - 1}))
    ws = torch.zeros(api.verify_sample_workspace_bytes(9), dtype=torch.uint8, device=DEV)
    for B in (2, 9, 1, 5, 9):
        p = torch.softmax(torch.randn((B, 2, 9000), generator=g, device=DEV), -1)
        q = torch.softmax(torch.randn((B, 1, 9000), generator=g, device=DEV), -1)
        d = torch.randint(0, 9000, (B, 1), generator=g, device=DEV).int()
        _verify(p, q, d, torch.rand((B, 2), generator=g, device=DEV), workspace=ws)
    assert api.check_device_error() == 0


@pytest.mark.parametrize("scale", [-0.05, 0.0, -1.0, 3e-4])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("min_mb", ["0", "80"])
def test_attention_scales(cuda_lib, monkeypatch, scale, dtype, min_mb):
    # the largest score is the smallest product where the scale is negative, and every key weighs the same at 0
    monkeypatch.setenv("QD_SHARED_MIN_MB", min_mb)
    g = _gen(25)
    hq, hkv, ps = 8, 2, 16
    rows, lens = [60, 2], [300, 90]
    kp, vp, pt = _cache(g, lens, hkv, ps)
    cu, seqs, seen = _pack(rows, lens)
    q = torch.randn((cu[-1], hq, D), generator=g, device=DEV).to(dtype)
    out = api.attn_prompt(q, kp, vp, pt, _ints(cu), _ints(lens), scale)
    _check_rows(out, q, kp, vp, pt, seqs, seen, range(0, 62, 3), scale=scale)
    lens = [300 + i for i in range(9)]
    kp, vp, pt = _cache(g, lens, hkv, ps, [(0, 16)] * 9)
    out = api.attn_decode_shared(q[:9], kp, vp, pt, _ints(lens), _ints([0, 9]), _ints([256]), scale)
    _check_rows(out, q[:9], kp, vp, pt, list(range(9)), lens, scale=scale)
    assert api.check_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_attention_of_many_short_sequences(cuda_lib, monkeypatch, dtype):
    # more sequences, and more groups, than a CTA has threads
    monkeypatch.setenv("QD_SHARED_MIN_MB", "0")
    g = _gen(26)
    hq, hkv, ps, B = 4, 2, 8, 1024
    rows = [(7 * i) % 4 for i in range(B)]
    lens = [n + (13 * i) % 50 for i, n in enumerate(rows)]
    kp, vp, pt = _cache(g, lens, hkv, ps)
    cu, seqs, seen = _pack(rows, lens)
    q = torch.randn((cu[-1], hq, D), generator=g, device=DEV).to(dtype)
    out = api.attn_prompt(q, kp, vp, pt, _ints(cu), _ints(lens), SCALE)
    _check_rows(out, q, kp, vp, pt, seqs, seen, list(range(0, cu[-1], 31)) + [cu[-1] - 1])
    members = [1 + i % 3 for i in range(B)]
    who = [i for i, n in enumerate(members) for _ in range(n)]
    starts = [0]
    for n in members:
        starts.append(starts[-1] + n)
    shared = [8 * (i % 5) for i in range(B)]
    lens = [shared[i] + (11 * b) % 20 for b, i in enumerate(who)]
    kp, vp, pt = _cache(g, lens, hkv, ps, [(i, shared[i] // ps) for i in who])
    q = torch.randn((len(who), hq, D), generator=g, device=DEV).to(dtype)
    out = api.attn_decode_shared(q, kp, vp, pt, _ints(lens), _ints(starts), _ints(shared), SCALE)
    pick = list(range(0, len(who), 31)) + [len(who) - 1]
    _check_rows(out, q, kp, vp, pt, list(range(len(who))), lens, pick)
    assert api.check_device_error() == 0


@pytest.mark.parametrize("op", ["prompt", "shared"])
def test_attention_calls_at_once_on_two_streams(cuda_lib, monkeypatch, op):
    monkeypatch.setenv("QD_SHARED_MIN_MB", "0")
    g = _gen(27)
    hq, hkv, ps, lens = 8, 2, 16, [2000, 1700, 1900]
    kp, vp, pt = _cache(g, lens, hkv, ps, [(0, 100)] * 3)
    ln, cu, sl = _ints(lens), _ints([0, 1, 2, 3]), _ints([1600])
    cu3 = _ints([0, 3])
    qs = [torch.randn((3, hq, D), generator=g, device=DEV) for _ in range(2)]
    nbytes = api.attn_prompt_workspace_bytes() if op == "prompt" else api.attn_shared_workspace_bytes(3, hq, hkv)
    ws = [torch.zeros(nbytes, dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs = [torch.zeros_like(qs[0]) for _ in range(2)]

    def call(i, **kw):
        if op == "prompt":
            return api.attn_prompt(qs[i], kp, vp, pt, cu, ln, SCALE, workspace=ws[i], **kw)
        return api.attn_decode_shared(qs[i], kp, vp, pt, ln, cu3, sl, SCALE, workspace=ws[i], **kw)

    want = [call(i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            call(i, out=outs[i], stream=streams[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    assert api.check_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_attention_of_one_head(cuda_lib, dtype):
    # heads of one: the stride between heads means nothing
    g = _gen(28)
    kp, vp, pt = _cache(g, [70], 1, 16)
    q = torch.randn((20, 3, 2 * D), generator=g, device=DEV).to(dtype)[:, ::2][:, :1, :D]
    out = api.attn_prompt(q, kp, vp, pt, _ints([0, 20]), _ints([70]), SCALE)
    _check_rows(out, q, kp, vp, pt, [0] * 20, list(range(51, 71)))
    with pytest.raises(ValueError):
        api.attn_prompt(torch.zeros((20, 3, 2 * D), dtype=dtype, device=DEV)[:, :2, :D], kp, vp, pt, _ints([0, 20]),
                        _ints([70]), SCALE)


# ------------------------------------------------------------------------------------------ page operations


def _page_cache(g, n_pages, ps, max_seqs, max_pages, layers=2, hkv=2, hd=8):
    k = [torch.randn((n_pages, hkv, ps, hd), generator=g, device=DEV).to(torch.bfloat16) for _ in range(layers)]
    v = [torch.randn((n_pages, hkv, ps, hd), generator=g, device=DEV).to(torch.bfloat16) for _ in range(layers)]
    return api.PageCache.empty(k, v, max_seqs, max_pages)


def _same(c, m, contents):
    """The device state equals the host model; the caches hold what the model's copies gave."""
    t, n, r = m.arrays()
    np.testing.assert_array_equal(c.page_table.cpu().numpy(), t)
    np.testing.assert_array_equal(c.seq_lens.cpu().numpy(), n)
    np.testing.assert_array_equal(c.refs.cpu().numpy(), r)
    for a, b in m.copies:
        for x in contents:
            x[b] = x[a]
    m.copies.clear()
    for x, y in zip(c.k_cache + c.v_cache, contents):
        assert torch.equal(x.cpu(), y)


@pytest.mark.parametrize("seed,n_pages,ps,max_seqs,hd", [(0, 40, 4, 9, 8), (1, 700, 16, 70, 16), (2, 33, 1, 5, 128),
                                                         (3, 20000, 3, 300, 8)])
def test_page_operations_against_host_lists(cuda_lib, seed, n_pages, ps, max_seqs, hd):
    g, r = _gen(seed), np.random.default_rng(seed)
    max_pages = 12
    c = _page_cache(g, n_pages, ps, max_seqs, max_pages, layers=1 if n_pages > 1000 else 3, hd=hd)
    m = ref.Pages(n_pages, ps, max_seqs, max_pages)
    contents = [x.cpu().clone() for x in c.k_cache + c.v_cache]
    refused = 0
    for step in range(40):
        op = ["extend", "fork", "extend", "trim", "compact"][step % 5] if step < 10 else r.choice(
            ["extend", "extend", "fork", "trim", "compact"])
        if op == "extend":
            n = np.where(r.random(max_seqs) < 0.5, r.integers(-1, 3 * ps + 2, max_seqs), 0).astype(np.int32)
            c.extend(_ints(n.tolist()))
            ok = m.extend(n.tolist())
        elif op == "fork":
            empty = [s for s in range(max_seqs) if not m.lens[s]]
            kids = r.permutation(empty)[:int(r.integers(0, len(empty) + 1))].tolist() if empty else []
            par = [int(x) for x in r.integers(0, max_seqs, len(kids))]
            c.fork(_ints(par), _ints(kids))
            ok = m.fork(par, kids)
        elif op == "trim":
            n = np.where(r.random(max_seqs) < 0.5, r.integers(-1, 4 * ps, max_seqs), -1).astype(np.int32)
            c.trim(_ints(n.tolist()))
            m.trim(n.tolist())
            ok = True
        else:
            assert int(c.compact()) == m.compact()
            ok = True
        assert api.check_device_error() == (0 if ok else 32), (step, op)
        refused += not ok
        _same(c, m, contents)
    assert refused < 35


def test_page_operations_refused_whole(cuda_lib):
    g = _gen(4)
    c = _page_cache(g, 10, 4, 6, 5)
    m = ref.Pages(10, 4, 6, 5)
    contents = [x.cpu().clone() for x in c.k_cache + c.v_cache]
    for n in ([9, 6, 0, 0, 0, 0],):
        c.extend(_ints(n))
        assert m.extend(n)
    for par, kid in (([0, 0], [2, 2]), ([0], [1]), ([6], [2]), ([-1], [2]), ([0], [6]), ([0], [-1]), ([2], [2]),
                     ([0, 1, 0], [2, 3, 1])):
        c.fork(_ints(par), _ints(kid))
        assert api.check_device_error() == 32
        _same(c, m, contents)
    for n in ([0, 0, 21, 0, 0, 0], [0, 15, 0, 0, 0, 0], [0, 0, 16, 8, 0, 0], [2**31 - 1, 1, 1, 1, 1, 1]):
        c.extend(_ints(n))
        assert api.check_device_error() == 32
        _same(c, m, contents)
    c.extend(_ints([0, 0, 16, 4, 0, 0]))     # exactly the pages that are left
    assert m.extend([0, 0, 16, 4, 0, 0]) and api.check_device_error() == 0
    _same(c, m, contents)
    # a sharer of a page that nobody may copy any more
    c.trim(_ints([0, -1, -1, -1, -1, -1]))
    m.trim([0, -1, -1, -1, -1, -1])
    c.fork(_ints([1, 1, 1]), _ints([0, 4, 5]))
    m.fork([1, 1, 1], [0, 4, 5])
    c.extend(_ints([2, 2, 0, 0, 2, 2]))      # three copies are needed, three pages free
    assert m.extend([2, 2, 0, 0, 2, 2]) and api.check_device_error() == 0
    _same(c, m, contents)


def test_page_copy(cuda_lib):
    g = _gen(11)
    for n_pages, ps, hd, layers in ((50, 16, 128, 3), (9, 5, 8, 70), (4, 129, 24, 1)):
        c = _page_cache(g, n_pages, ps, 1, 1, layers=layers, hd=hd)
        want = [x.clone() for x in c.k_cache + c.v_cache]
        ids = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
        n = n_pages // 2
        src, dst = ids[:n].clone(), ids[n:2 * n].clone()
        src[0] = -1                      # skipped
        if n > 2:
            src[2] = src[1]              # one source twice
        c.copy(src, dst)
        for x in want:
            x[dst[1:].long()] = x[src[1:].long()]
        assert all(torch.equal(x, y) for x, y in zip(c.k_cache + c.v_cache, want))
        assert api.check_device_error() == 0
        c.copy(_ints([n_pages]), _ints([0]))
        assert api.check_device_error() == 1
        assert all(torch.equal(x, y) for x, y in zip(c.k_cache + c.v_cache, want))


def test_page_operations_in_a_graph(cuda_lib):
    g = _gen(12)
    c = _page_cache(g, 64, 4, 8, 8)
    m = ref.Pages(64, 4, 8, 8)
    contents = [x.cpu().clone() for x in c.k_cache + c.v_cache]
    grow, par, kid, cut = _ints([0] * 8), _ints([0, 0]), _ints([3, 5]), _ints([-1] * 8)
    live = torch.zeros(1, dtype=torch.int32, device=DEV)
    c.extend(_ints([6, 9, 0, 0, 0, 0, 0, 0]))
    m.extend([6, 9, 0, 0, 0, 0, 0, 0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.fork(par, kid)
        c.extend(grow)
        c.trim(cut)
        c.compact(live)
    for n, t in (([1] * 8, [-1, 0, -1, 0, -1, 0, -1, -1]), ([3, 0, 1, 0, 0, 2, 0, 0], [5, -1, -1, 0, 0, 0, -1, 2])):
        grow.copy_(_ints(n))
        cut.copy_(_ints(t))
        graph.replay()
        m.fork([0, 0], [3, 5])
        assert m.extend(n)
        m.trim(t)
        assert int(live) == m.compact()
        _same(c, m, contents)
    assert api.check_device_error() == 0


def test_page_operations_of_many_sequences(cuda_lib):
    # as many sequences as there may be, most of them sharers of three pages, extended in one call
    g, r = _gen(13), np.random.default_rng(13)
    n = 2048
    c = _page_cache(g, 5000, 4, n, 6, layers=1)
    m = ref.Pages(5000, 4, n, 6)
    contents = [x.cpu().clone() for x in c.k_cache + c.v_cache]
    start = [6, 9, 3] + [0] * (n - 3)
    kids = r.permutation(np.arange(3, n))[:1500].tolist()
    par = r.integers(0, 3, 1500).tolist()
    for grow in (start, np.where(r.random(n) < 0.7, r.integers(0, 3, n), 0).tolist(), r.integers(0, 2, n).tolist()):
        c.extend(_ints(grow))
        assert m.extend(grow) and api.check_device_error() == 0
        _same(c, m, contents)
        if grow is start:
            c.fork(_ints(par), _ints(kids))
            assert m.fork(par, kids)


# -------------------------------------------------------------------------------------- sampled verification


def _verify(p, q, draft, u, n_draft=None, steps=12, start=None, workspace=None):
    B, k, V = p.shape
    step = start.clone() if start is not None else torch.zeros(B, dtype=torch.int32, device=DEV)
    tok, pos = torch.full((B,), -5, dtype=torch.int32, device=DEV), torch.arange(B, dtype=torch.int32, device=DEV)
    out = torch.full((B, steps), -1, dtype=torch.int32, device=DEV)
    first, n0 = step.tolist(), pos.tolist()
    m = api.verify_sample(p, q, draft, u, tok, pos, step, out, n_draft=n_draft, workspace=workspace)
    host = [x.double().cpu().numpy() if x is not None else None for x in (p, q, u)]
    d = draft.cpu().numpy() if draft is not None else np.zeros((B, 0), int)
    err = 0
    for b in range(B):
        nd = k - 1 if n_draft is None else int(n_draft[b])
        if nd < 0 or nd > k - 1:
            nd, err = min(max(nd, 0), k - 1), err | 2
        wm, wt = ref.verify(host[0][b], host[1][b] if k > 1 else host[0][b], d[b], host[2][b], nd)
        assert (int(m[b]), int(tok[b])) == (wm, wt), b
        line = [int(x) for x in d[b, :wm]] + [wt]
        want = [-1] * steps
        for i, t in enumerate(line):
            if 0 <= first[b] + i < steps:
                want[first[b] + i] = t
            else:
                err |= 8
        assert out[b].tolist() == want, b
        assert int(pos[b]) == n0[b] + wm + 1 and int(step[b]) == first[b] + wm + 1
    return m, tok, err


@pytest.mark.parametrize("B,k,V,near", [(1, 1, 1, 0.5), (1, 4, 151936, 0.3), (3, 2, 50, 1.0), (5, 8, 4096, 0.2),
                                        (64, 5, 5003, 0.5), (2, 40, 1025, 0.05), (9, 3, 16385, 2.0), (4, 6, 7, 0.5)])
def test_verify_sample(cuda_lib, B, k, V, near):
    g = _gen(B * k + V)
    z = torch.randn((B, max(1, k), V), generator=g, device=DEV) * 2
    p = torch.softmax(z + near * torch.randn((B, k, V), generator=g, device=DEV), -1)
    q = torch.softmax(z[:, :k - 1], -1).contiguous() if k > 1 else None
    draft = torch.multinomial(q.flatten(0, 1), 1, generator=g).view(B, k - 1).int() if k > 1 else None
    for _ in range(4):
        u = torch.rand((B, k), generator=g, device=DEV)
        _verify(p, q, draft, u, steps=k + 3)
    assert api.check_device_error() == 0


def test_verify_sample_padded_rows_ragged_drafts_and_bad_drafts(cuda_lib):
    g = _gen(31)
    B, k, V = 6, 4, 1003
    pw = torch.softmax(torch.randn((B, k, 1100), generator=g, device=DEV), -1)
    qw = torch.softmax(torch.randn((B, k - 1, 1101), generator=g, device=DEV), -1)
    draft = torch.randint(0, V, (B, k - 1), generator=g, device=DEV).int()
    draft[2, 0], draft[3, 1] = V, -1
    u = torch.rand((B, k), generator=g, device=DEV) * 0.5
    n = _ints([0, 1, 3, 3, 4, -2])
    start = _ints([0, 3, 0, 11, 0, 0])
    _, _, err = _verify(pw[..., :V], qw[..., :V], draft, u, n_draft=n, start=start)
    assert api.check_device_error() == err and err & 2


def test_verify_sample_borders(cuda_lib):
    # probabilities that are multiples of 2^-10, so every sum is exact and a border can be met exactly
    V = 1024
    even = torch.full((1, 1, V), 1 / V, device=DEV)
    for u in (0.0, 1 / V, 5 / V, 0.5, 1 - 1 / V, 1 - 2.0 ** -24):
        _, tok, _ = _verify(even, None, None, torch.full((1, 1), u, device=DEV))
        assert int(tok) == min(int(u * V), V - 1)
    # u q(d) == p(d) is a rejection; below it, acceptance
    p = torch.zeros((1, 2, V), device=DEV)
    q = torch.zeros((1, 1, V), device=DEV)
    p[0, 0, 3], p[0, 0, 9], p[0, 1, 100], q[0, 0, 3], q[0, 0, 7] = 0.25, 0.75, 1.0, 0.5, 0.5
    d = _ints([[3]])
    for u0, want in ((0.5, (0, 9)), (0.5 - 2.0 ** -24, (1, 100)), (0.0, (1, 100))):
        m, tok, _ = _verify(p, q, d, torch.tensor([[u0, 0.3]], device=DEV))
        assert (int(m), int(tok)) == want
    # a draft with q = 0: accepted if p has any mass there
    for tokn, want in ((9, 1), (11, 0)):
        m, _, _ = _verify(p, q, _ints([[tokn]]), torch.tensor([[0.9, 0.3]], device=DEV))
        assert int(m) == want
    # p == q and still rejected (u = 1): drawn from p
    m, tok, _ = _verify(torch.cat([q, q], 1), q, d, torch.tensor([[1.0, 0.75]], device=DEV))
    assert (int(m), int(tok)) == (0, 7)
    assert api.check_device_error() == 0


def test_verify_sample_entries_that_are_not_finite(cuda_lib):
    V = 5000
    p = torch.zeros((3, 1, V), device=DEV)
    p[0, 0, 40], p[0, 0, 41], p[0, 0, 4000] = math.nan, math.inf, 0.5
    p[1, 0, 17] = -1.0
    p[2] = math.nan
    _, tok, _ = _verify(p, None, None, torch.full((3, 1), 0.4, device=DEV))
    assert tok.tolist() == [4000, 0, 0]
    assert api.check_device_error() == 4


def test_verify_sample_of_many_sequences(cuda_lib):
    g = _gen(34)
    B, k, V = 1500, 3, 37
    p = torch.softmax(torch.randn((B, k, V), generator=g, device=DEV), -1)
    q = torch.softmax(torch.randn((B, k - 1, V), generator=g, device=DEV), -1)
    draft = torch.randint(0, V, (B, k - 1), generator=g, device=DEV).int()
    _verify(p, q, draft, torch.rand((B, k), generator=g, device=DEV))
    assert api.check_device_error() == 0


def test_verify_sample_in_a_graph(cuda_lib):
    g = _gen(33)
    B, k, V = 4, 3, 9001
    p = torch.softmax(torch.randn((B, k, V), generator=g, device=DEV), -1)
    q = torch.softmax(torch.randn((B, k - 1, V), generator=g, device=DEV), -1)
    draft = torch.randint(0, V, (B, k - 1), generator=g, device=DEV).int()
    u = torch.rand((B, k), generator=g, device=DEV)
    ws = torch.zeros(api.verify_sample_workspace_bytes(B), dtype=torch.uint8, device=DEV)
    tok, pos, step, m = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(4))
    out = torch.full((B, 16), -1, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.verify_sample(p, q, draft, u, tok, pos, step, out, n_accept=m, workspace=ws)
    total = np.zeros(B, int)
    for _ in range(4):
        u.copy_(torch.rand((B, k), generator=g, device=DEV))
        graph.replay()
        for b in range(B):
            want = ref.verify(p[b].double().cpu().numpy(), q[b].double().cpu().numpy(), draft[b].cpu().numpy(),
                              u[b].double().cpu().numpy(), k - 1)
            assert (int(m[b]), int(tok[b])) == want
            total[b] += want[0] + 1
    assert step.tolist() == total.tolist() and api.check_device_error() == 0


# ------------------------------------------------------------------------------------------- all of them, as used


@pytest.mark.parametrize("min_mb", ["0", "80"])
def test_a_serving_round(cuda_lib, monkeypatch, min_mb):
    """Two prompts in one call, each forked to samples, decode over the shared prefixes, drafts verified,
    rejected tokens given back, the cache compacted; attention before and after compaction is the same."""
    monkeypatch.setenv("QD_SHARED_MIN_MB", min_mb)
    g = _gen(40)
    hq, hkv, ps, V = 8, 2, 16, 600
    n_pages, max_seqs, max_pages = 200, 12, 20
    k = [torch.full((n_pages, hkv, ps, D), math.nan, dtype=torch.bfloat16, device=DEV)]
    v = [torch.full((n_pages, hkv, ps, D), math.nan, dtype=torch.bfloat16, device=DEV)]
    c = api.PageCache.empty(k, v, max_seqs, max_pages)

    def write(old, new):   # the tokens' K/V, as the projections would
        for s in range(max_seqs):
            for t in range(old[s], new[s]):
                page = int(c.page_table[s, t // ps])
                for x in (k[0], v[0]):
                    x[page, :, t % ps] = torch.randn((hkv, D), generator=g, device=DEV).to(torch.bfloat16)

    # other sequences come and go, so that the pages are scattered
    c.extend(_ints([0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 50, 70]))
    lens0 = c.seq_lens.tolist()
    c.extend(_ints([75, 0, 0, 0, 0, 133] + [0] * 6))
    c.trim(_ints([-1] * 10 + [0, 0]))
    lens0[10] = lens0[11] = 0
    now = c.seq_lens.tolist()
    write(lens0, now)
    rows = [now[0], now[5]]
    table2, lens2 = c.page_table[[0, 5]].contiguous(), c.seq_lens[[0, 5]].contiguous()
    cu, seqs, seen = _pack(rows, rows)
    q = torch.randn((sum(rows), hq, D), generator=g, device=DEV).to(torch.bfloat16)
    out = api.attn_prompt(q, k[0], v[0], table2, _ints(cu), lens2, SCALE)
    _check_rows(out, q, k[0], v[0], table2, seqs, seen, range(0, sum(rows), 11))

    c.fork(_ints([0, 0, 0, 0, 5, 5]), _ints([1, 2, 3, 4, 6, 7]))
    kd = 3                                           # drafts per sequence
    before = c.seq_lens.tolist()
    c.extend(_ints([kd + 1] * 8 + [0] * 4))
    write(before, c.seq_lens.tolist())
    cu_g, shared = _ints([0, 5, 8]), _ints([75 // ps * ps, 133 // ps * ps])

    def decode():
        qd = torch.randn((8, hq, D), generator=_gen(41), device=DEV)
        t, n = c.page_table[:8].contiguous(), c.seq_lens[:8].contiguous()
        o = api.attn_decode_shared(qd, k[0], v[0], t, n, cu_g, shared, SCALE)
        _check_rows(o, qd, k[0], v[0], t, list(range(8)), n.tolist())
        return o

    decode()
    p = torch.softmax(torch.randn((8, kd + 1, V), generator=g, device=DEV), -1)
    qd = torch.softmax(torch.randn((8, kd, V), generator=g, device=DEV), -1)
    draft = torch.multinomial(qd.flatten(0, 1), 1, generator=g).view(8, kd).int()
    m, _, _ = _verify(p, qd, draft, torch.rand((8, kd + 1), generator=g, device=DEV) * 0.7)
    keep = torch.full((max_seqs,), -1, dtype=torch.int32, device=DEV)
    keep[:8] = torch.tensor(before[:8], dtype=torch.int32, device=DEV) + m + 1
    c.trim(keep)
    assert c.seq_lens.tolist()[:8] == [b + int(x) + 1 for b, x in zip(before, m)]
    a = decode()
    n = int(c.compact())
    assert n == int((c.refs > 0).sum()) and int(c.page_table.max()) == n - 1
    assert torch.equal(a, decode())
    c.trim(_ints([0] * max_seqs))
    assert int(c.refs.abs().sum()) == 0 and int(c.page_table.max()) == -1
    assert api.check_device_error() == 0
