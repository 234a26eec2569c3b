"""Attention over a sliding window and first tokens that stay visible, and the weights it gives to the keys, on the
GPU against plain 64-bit implementations."""
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
POS, PAGE = 2, 1
DTYPES = [torch.float32, torch.bfloat16]


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _q(g, n, hq, dtype, scale=1.0):
    return (torch.randn((n, hq, D), generator=g, device=DEV) * scale).to(dtype)


# ------------------------------------------------------------------------------------------------- single tokens


def _check_decode(out, q, kp, vp, pt, lens, window, sinks, scale=SCALE, sums=None, before=None, only=None):
    bf16 = q.dtype == torch.bfloat16
    out, qd = out.double().cpu(), q.double().cpu()
    for b, n in enumerate(lens):
        if only is not None and b not in only:
            continue
        k, v = ref.tokens(kp, pt[b], n), ref.tokens(vp, pt[b], n)
        see = ref.visible(n - 1, n, window, sinks)
        want, w, mag, dot = ref.attend(qd[b], k, v, see, scale)
        m = int(see.sum())
        tol = ref.out_bound(want, mag, dot, m, bf16, 2 if bf16 else 3)
        err = (out[b] - want).abs()
        assert bool((err <= tol).all()), (b, n, float((err / tol).max()))
        if sums is not None:
            got, old = sums[b].double().cpu(), before[b].double().cpu()
            assert torch.equal(got[:, n:], old[:, n:]) and torch.equal(got[:, :n][:, ~see], old[:, :n][:, ~see])
            total = old[:, :n] + w
            tol = ref.weight_bound(dot, m) * w + 2.0 ** -23 * total + 1e-30
            err = (got[:, :n] - total).abs()
            assert bool((err <= tol).all()), (b, n, float((err / tol).max()))


DECODE = [   # lengths, q heads, kv heads, page size, window, first tokens
    ([1], 4, 2, 16, 1, 0),
    ([0, 1, 2, 3], 4, 2, 16, 2, 1),
    ([17, 300, 64, 5], 8, 8, 16, 16, 4),
    ([100, 101, 102, 103, 104], 8, 1, 16, 100, 3),
    ([1000, 333], 32, 8, 16, 128, 130),
    ([777, 1500, 15], 8, 2, 7, 333, 5),
    ([2000, 1], 16, 2, 24, 700, 64),
    ([900], 8, 2, 256, 64, 300),
    ([50, 60], 2, 2, 1, 13, 2),
    ([5000], 8, 1, 128, ALL, 0),
    ([20000], 16, 8, 16, 1024, 4),
    ([4000, 12, 900], 4, 4, 64, ALL, 7),
    ([70, 33], 4, 2, 16, 5, 1000),             # more first tokens than there are
    ([130] * 40, 32, 8, 16, 96, 4),
    ([2500, 1300, 2049] * 6, 32, 8, 16, 2100, 0),      # many pairs, each in a few long splits
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens,hq,hkv,ps,window,sinks", DECODE)
def test_decode(cuda_lib, lens, hq, hkv, ps, window, sinks, dtype):
    g = _gen(sum(lens) + hq)
    kp, vp, pt = ref.make_cache(g, lens, hkv, ps)
    cap = pt.shape[1] * ps
    q = _q(g, len(lens), hq, dtype)
    ws = torch.zeros(api.attn_decode_window_workspace_bytes(len(lens), hq, hkv, min(window + sinks, cap)),
                     dtype=torch.uint8, device=DEV)
    plain = api.attn_decode_window(q, kp, vp, pt, _ints(lens), SCALE, window, sinks, workspace=ws)
    _check_decode(plain, q, kp, vp, pt, lens, window, sinks)
    before = torch.rand((len(lens), hkv, cap), generator=g, device=DEV) * 0.1
    sums = before.clone()
    out = api.attn_decode_window(q, kp, vp, pt, _ints(lens), SCALE, window, sinks, key_weights=sums, workspace=ws)
    assert torch.equal(out, plain)             # asking for the weights changes nothing else
    _check_decode(out, q, kp, vp, pt, lens, window, sinks, sums=sums, before=before)
    again = before.clone()                     # the workspace is left ready, and the order of sums fixed
    assert torch.equal(out, api.attn_decode_window(q, kp, vp, pt, _ints(lens), SCALE, window, sinks, key_weights=again))
    assert torch.equal(again, sums)
    assert api.check_device_error() == 0


@pytest.mark.parametrize("seed", range(6))
def test_decode_ragged(cuda_lib, seed):
    g, r = _gen(seed), np.random.default_rng(seed)
    hq, hkv = [(32, 8), (8, 8), (16, 2), (4, 2), (8, 1), (1, 1)][seed]
    B = int(r.integers(1, 24))
    lens = [int(x) for x in 2 ** r.uniform(0, 13, B)]
    window, sinks, ps = int(2 ** r.uniform(0, 12)), int(r.integers(0, 200)), int(r.choice([7, 16, 24, 128]))
    dtype = DTYPES[seed % 2]
    kp, vp, pt = ref.make_cache(g, lens, hkv, ps)
    q = _q(g, B, hq, dtype, 1 + 5 * (seed % 3))
    sums = torch.zeros((B, hkv, pt.shape[1] * ps), device=DEV)
    before = sums.clone()
    out = api.attn_decode_window(q, kp, vp, pt, _ints(lens), SCALE, window, sinks, key_weights=sums)
    _check_decode(out, q, kp, vp, pt, lens, window, sinks, sums=sums, before=before)
    assert api.check_device_error() == 0


def test_decode_equals_the_other_decode_attention(cuda_lib):
    g = _gen(3)
    lens = [1, 700, 64, 2100]
    kp, vp, pt = ref.make_cache(g, lens, 2, 16)
    q = _q(g, 4, 8, torch.float32)
    a = api.attn_decode_window(q, kp, vp, pt, _ints(lens), SCALE)
    b = api.attn_decode_paged(q, kp, vp, pt, _ints(lens), SCALE)
    # (that one has q and the weights in two parts)
    assert float((a - b).abs().max() / b.abs().max()) < 2.0 ** -13


@pytest.mark.parametrize("scale", [-SCALE, 0.0, 1.0])
def test_decode_scales(cuda_lib, scale):
    g = _gen(4)
    lens = [300, 40]
    kp, vp, pt = ref.make_cache(g, lens, 2, 16)
    for dtype in DTYPES:
        q = _q(g, 2, 8, dtype)
        sums = torch.zeros((2, 2, pt.shape[1] * 16), device=DEV)
        out = api.attn_decode_window(q, kp, vp, pt, _ints(lens), scale, 100, 3, key_weights=sums)
        _check_decode(out, q, kp, vp, pt, lens, 100, 3, scale, sums, torch.zeros_like(sums))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", DTYPES)
def test_decode_hidden_values(cuda_lib, dtype, bad):
    # tokens between the first ones and the window, and slots behind the last token, hold anything
    g = _gen(5)
    lens, window, sinks = [500, 90, 33], 70, 9
    kp, vp, pt = ref.make_cache(g, lens, 2, 16, room=20)
    q = _q(g, 3, 8, dtype)
    clean_k, clean_v = kp.clone(), vp.clone()
    for b, n in enumerate(lens):
        for t in list(range(min(sinks, n), max(sinks, n - window))) + list(range(n, -(-n // 16) * 16)):
            kp[int(pt[b, t // 16]), :, t % 16] = bad
            vp[int(pt[b, t // 16]), :, t % 16] = bad
    sums = torch.zeros((3, 2, pt.shape[1] * 16), device=DEV)
    out = api.attn_decode_window(q, kp, vp, pt, _ints(lens), SCALE, window, sinks, key_weights=sums)
    _check_decode(out, q, clean_k, clean_v, pt, lens, window, sinks, sums=sums, before=torch.zeros_like(sums))


@pytest.mark.parametrize("dtype", DTYPES)
def test_decode_visible_nan_and_infinity(cuda_lib, dtype):
    g = _gen(6)
    lens = [2000, 2000]
    kp, vp, pt = ref.make_cache(g, lens, 2, 16)
    q = _q(g, 2, 8, dtype)
    vp[int(pt[0, 100]), 1, 3, 7] = math.nan            # token 1603
    vp[int(pt[0, 101]), 1, 3, 9] = math.inf
    kp[int(pt[1, 100]), 0, 3, 7] = math.nan
    sums = torch.zeros((2, 2, 2000), device=DEV)
    out = api.attn_decode_window(q, kp, vp, pt, _ints(lens), SCALE, 600, 4, key_weights=sums)
    assert bool(out[0, 4:, 7].isnan().all()) and not bool(out[0, 4:, 9].isfinite().any())
    assert int((~out[0].isfinite()).sum()) == 8 and bool(out[1, :4].isnan().all()) and bool(out[1, 4:].isfinite().all())
    assert bool(sums[1, 0, 1400:].isnan().all()) and bool(sums[1, 0, 4:1400].eq(0).all())
    assert bool(sums[0].isfinite().all()) and bool(sums[1, 1].isfinite().all())
    hidden = api.attn_decode_window(q, kp, vp, pt, _ints(lens), SCALE, 300, 4)
    assert bool(hidden.isfinite().all())
    kp[int(pt[1, 100]), 0, 3, 7] = 0
    q[1, 4:] = 0
    kp[int(pt[1, 0]), 1, 0, 0] = -math.inf              # 0 * inf: NaN as the formula's
    assert bool(api.attn_decode_window(q, kp, vp, pt, _ints(lens), SCALE, 600, 4)[1, 4:].isnan().all())


def test_decode_large_scores(cuda_lib):
    g = _gen(8)
    lens = [900, 2500]
    kp, vp, pt = ref.make_cache(g, lens, 2, 16)
    q = _q(g, 2, 8, torch.bfloat16, 40)
    sums = torch.zeros((2, 2, pt.shape[1] * 16), device=DEV)
    out = api.attn_decode_window(q, kp, vp, pt, _ints(lens), SCALE, 800, 4, key_weights=sums)
    _check_decode(out, q, kp, vp, pt, lens, 800, 4, sums=sums, before=torch.zeros_like(sums))


def test_decode_strided_q_and_broken_lengths(cuda_lib):
    g = _gen(9)
    lens = [40, 33, 5]
    kp, vp, pt = ref.make_cache(g, lens, 2, 16)
    qkv = _q(g, 3, 12, torch.float32)
    out = torch.full((3, 8, D), 7.0, device=DEV)
    sums = torch.full((3, 2, 48), 7.0, device=DEV)
    before = sums.clone()
    api.attn_decode_window(qkv[:, :8], kp, vp, pt, _ints([40, 49, 5]), SCALE, 20, 1, key_weights=sums, out=out)
    assert api.check_device_error() == POS
    _check_decode(out, qkv[:, :8], kp, vp, pt, lens, 20, 1, sums=sums, before=before, only=[0, 2])
    assert bool((out[1] == 7).all()) and bool((sums[1] == 7).all())
    api.attn_decode_window(qkv[:, :8], kp, vp, pt, _ints([40, -1, 5]), SCALE, 20, 1, key_weights=sums, out=out)
    assert api.check_device_error() == POS and bool((out[1] == 7).all()) and bool((sums[1] == 7).all())
    pt[0, 2] = kp.shape[0]
    api.attn_decode_window(qkv[:, :8], kp, vp, pt, _ints(lens), SCALE, 20, 1, out=out)
    assert api.check_device_error() == PAGE


def test_decode_weights_add_up_over_calls(cuda_lib):
    g = _gen(10)
    lens = [130, 50]
    kp, vp, pt = ref.make_cache(g, lens, 2, 16)
    sums = torch.zeros((2, 2, pt.shape[1] * 16), device=DEV)
    for i in range(5):
        api.attn_decode_window(_q(g, 2, 8, torch.bfloat16), kp, vp, pt, _ints(lens), SCALE, 64, 2, key_weights=sums)
    total = sums.double().sum(-1)
    assert bool((total - 5 * 4).abs().max() < 5 * 4 * 2.0 ** -16)      # every row's weights are 1 together


def test_decode_in_graphs_that_share_a_workspace(cuda_lib):
    g = _gen(11)
    hq, hkv = 8, 2
    ws = torch.zeros(api.attn_decode_window_workspace_bytes(5, hq, hkv, 1008), dtype=torch.uint8, device=DEV)
    runs = []
    for B, dtype in ((5, torch.float32), (2, torch.bfloat16)):
        kp, vp, pt = ref.make_cache(g, [1000] * B, hkv, 16)
        r = dict(kp=kp, vp=vp, pt=pt, q=_q(g, B, hq, dtype), lens=_ints([1000] * B),
                 sums=torch.zeros((B, hkv, pt.shape[1] * 16), device=DEV), out=torch.empty((B, hq, D), dtype=dtype, device=DEV))

        def call(r=r):
            api.attn_decode_window(r["q"], r["kp"], r["vp"], r["pt"], r["lens"], SCALE, 300, 4, key_weights=r["sums"],
                                   out=r["out"], workspace=ws)

        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        runs.append((r, graph))
    for step in range(3):
        for r, graph in runs:
            B = r["q"].shape[0]
            lens = [int(x) for x in np.random.default_rng(step).integers(0, 1001, B)]
            r["lens"].copy_(_ints(lens))
            r["q"].copy_(torch.randn(r["q"].shape, generator=g, device=DEV))
            r["sums"].zero_()
            graph.replay()
            _check_decode(r["out"], r["q"], r["kp"], r["vp"], r["pt"], lens, 300, 4, sums=r["sums"],
                          before=torch.zeros_like(r["sums"]))
    assert api.check_device_error() == 0


def test_decode_on_two_streams_at_once(cuda_lib):
    g = _gen(12)
    lens = [3000] * 8
    kp, vp, pt = ref.make_cache(g, lens, 2, 16)
    q = [_q(g, 8, 8, torch.float32) for _ in range(2)]
    n = _ints(lens)
    want = [api.attn_decode_window(x, kp, vp, pt, n, SCALE, 2000, 4) for x in q]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(20):
        for x, s in zip(q, streams):
            s.wait_stream(torch.cuda.current_stream())
            got.append(api.attn_decode_window(x, kp, vp, pt, n, SCALE, 2000, 4, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want[i % 2]) for i, a in enumerate(got))


def test_decode_many_sequences(cuda_lib):
    # more (sequence, kv head) pairs than there are tickets
    g, r = _gen(13), np.random.default_rng(13)
    B = 2100
    lens = [int(x) for x in r.integers(0, 60, B)]
    kp, vp, pt = ref.make_cache(g, lens, 2, 16)
    q = _q(g, B, 4, torch.bfloat16)
    sums = torch.zeros((B, 2, pt.shape[1] * 16), device=DEV)
    out = api.attn_decode_window(q, kp, vp, pt, _ints(lens), SCALE, 30, 2, key_weights=sums)
    _check_decode(out, q, kp, vp, pt, lens, 30, 2, sums=sums, before=torch.zeros_like(sums),
                  only=set(r.choice(B, 60).tolist()) | {0, B - 1})
    assert api.attn_decode_window(q[:0], kp, vp, pt[:0], _ints([]), SCALE).shape == (0, 4, D)
    assert api.check_device_error() == 0


# --------------------------------------------------------------------------------------------------- packed rows


def _pack(rows, lens):
    cu = [0]
    for n in rows:
        cu.append(cu[-1] + n)
    return cu, [b for b, n in enumerate(rows) for _ in range(n)], [m - n + j for n, m in zip(rows, lens) for j in range(n)]


def _check_prompt(out, q, kp, vp, pt, lens, seqs, at, window, sinks, scale=SCALE, rows=None):
    bf16 = q.dtype == torch.bfloat16
    out, q = out.double().cpu(), q.double().cpu()
    kv = {}
    for r in range(len(seqs)) if rows is None else rows:
        b, n = seqs[r], at[r] + 1
        if b not in kv:
            kv[b] = ref.tokens(kp, pt[b], lens[b]), ref.tokens(vp, pt[b], lens[b])
        see = ref.visible(at[r], max(n, 0), window, sinks)
        want, _, mag, dot = ref.attend(q[r], kv[b][0][:max(n, 0)], kv[b][1][:max(n, 0)], see, scale)
        tol = ref.out_bound(want, mag, dot, int(see.sum()), bf16, 1 if bf16 else 3)
        err = (out[r] - want).abs()
        assert bool((err <= tol).all()), (r, b, n, float((err / tol).max()))


def _pick(n, r):
    some = r.choice(n, min(60, n), replace=False).tolist()
    return sorted(set(range(min(n, 20))) | set(range(max(0, n - 10), n)) | set(some))


PROMPT = [   # rows, lengths, q heads, kv heads, page size, window, first tokens
    ([1], [1], 4, 2, 16, 1, 0),
    ([1, 1, 1], [1, 17, 300], 8, 8, 16, 16, 4),
    ([128], [128], 4, 4, 16, 1, 0),
    ([129, 0, 127], [129, 40, 127], 4, 2, 32, 64, 3),
    ([64, 65, 3, 31], [64, 65, 1000, 331], 32, 8, 16, 100, 130),
    ([300, 17], [300, 900], 16, 2, 64, 200, 5),
    ([33, 70], [729, 470], 4, 2, 7, 128, 128),
    ([40, 200], [40, 1500], 8, 2, 24, 129, 1),
    ([16, 20], [5, 20], 4, 2, 16, 6, 2),        # rows before position 0 see nothing
    ([9, 4], [0, 0], 4, 1, 16, 10, 4),
    ([1], [5000], 8, 1, 128, 700, 4),
    ([600], [2100], 8, 2, 256, 256, 256),
    ([2, 0, 0, 1], [2, 0, 7, 257], 2, 2, 1, 33, 2),
    ([700], [700], 8, 2, 16, 127, 0),
    ([1500], [3000], 4, 4, 16, 384, 64),        # one q head a kv head: tiles of 128 tokens
    ([260], [5000], 8, 1, 16, 1111, 513),
    ([90, 20], [150, 45], 8, 2, 16, ALL, 0),
    ([90, 20], [150, 45], 8, 2, 16, 20, 1000),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,lens,hq,hkv,ps,window,sinks", PROMPT)
def test_prompt(cuda_lib, rows, lens, hq, hkv, ps, window, sinks, dtype):
    g = _gen(sum(rows) + hq)
    kp, vp, pt = ref.make_cache(g, lens, hkv, ps)
    cu, seqs, at = _pack(rows, lens)
    q = _q(g, cu[-1], hq, dtype)
    ws = torch.zeros(api.attn_prompt_workspace_bytes(), dtype=torch.uint8, device=DEV)
    args = (q, kp, vp, pt, _ints(cu), _ints(lens), SCALE, window, sinks)
    first = api.attn_prompt_window(*args, workspace=ws)
    assert torch.equal(first, api.attn_prompt_window(*args, workspace=ws))
    _check_prompt(first, q, kp, vp, pt, lens, seqs, at, window, sinks, rows=_pick(cu[-1], np.random.default_rng(0)))
    assert api.check_device_error() == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("seed", range(10))
def test_prompt_ragged(cuda_lib, seed, dtype):
    g, r = _gen(60 + seed), np.random.default_rng(seed)
    hq, hkv = [(8, 1), (4, 4), (32, 8), (16, 2), (8, 8)][seed % 5]
    n = int(r.integers(1, 40))
    lens = [int(x) for x in 2 ** r.uniform(0, 12.5, n)]
    rows = [min(m, int(x)) for m, x in zip(lens, 2 ** r.uniform(0, 11, n))]
    window, sinks, ps = int(2 ** r.uniform(0, 11)), int(r.integers(0, 300)), int(r.choice([7, 16, 24, 64, 128]))
    kp, vp, pt = ref.make_cache(g, lens, hkv, ps)
    cu, seqs, at = _pack(rows, lens)
    q = _q(g, cu[-1], hq, dtype, 1 + 6 * (seed % 3))
    args = (q, kp, vp, pt, _ints(cu), _ints(lens), SCALE, window, sinks)
    ws = torch.zeros(api.attn_prompt_workspace_bytes(), dtype=torch.uint8, device=DEV)
    first = api.attn_prompt_window(*args, workspace=ws)
    for _ in range(5):
        assert torch.equal(first, api.attn_prompt_window(*args, workspace=ws))
    _check_prompt(first, q, kp, vp, pt, lens, seqs, at, window, sinks, rows=_pick(cu[-1], r))
    assert api.check_device_error() == 0


def _gone(pt, kp, vp, lens, first_at, window, sinks, ps, bad, drop):
    """Everything that no row from slot first_at on sees holds `bad`; with `drop`, whole pages of it are not named."""
    for b, n in enumerate(lens):
        t = torch.arange(-(-n // ps) * ps)
        hidden = ((t >= sinks) & (t <= first_at[b] - window)) | (t >= n)
        for i in range(len(t) // ps):
            h, page = hidden[i * ps:(i + 1) * ps].to(DEV), int(pt[b, i])
            kp[page, :, h] = bad
            vp[page, :, h] = bad
            if drop and bool(h.all()):
                pt[b, i] = [-1, kp.shape[0] + 5][i % 2]


@pytest.mark.parametrize("ps", [16, 64, 24])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", DTYPES)
def test_prompt_hidden_values_and_pages(cuda_lib, dtype, bad, ps):
    g = _gen(6)
    rows, lens, hq, hkv, window, sinks = [90, 20, 1], [1150, 445, 700], 8, 2, 200, 20
    kp, vp, pt = ref.make_cache(g, lens, hkv, ps)
    cu, seqs, at = _pack(rows, lens)
    q = _q(g, cu[-1], hq, dtype)
    ck, cv, cpt = kp.clone(), vp.clone(), pt.clone()
    _gone(pt, kp, vp, lens, [m - n for n, m in zip(rows, lens)], window, sinks, ps, bad, True)
    out = api.attn_prompt_window(q, kp, vp, pt, _ints(cu), _ints(lens), SCALE, window, sinks)
    _check_prompt(out, q, ck, cv, cpt, lens, seqs, at, window, sinks)
    assert api.check_device_error() == 0
    last = [cu[1] - 1, cu[2] - 1, cu[3] - 1]         # the same for single tokens
    one = api.attn_decode_window(q[last].contiguous(), kp, vp, pt, _ints(lens), SCALE, window, sinks)
    _check_decode(one, q[last], ck, cv, cpt, lens, window, sinks)
    assert api.check_device_error() == 0


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", DTYPES)
def test_prompt_value_reaches_the_rows_that_see_it(cuda_lib, dtype, what):
    # tokens that leave the window of some rows of a tile, and one of the first tokens
    g = _gen(7)
    rows, lens, hq, hkv, window, sinks = [400], [900], 4, 2, 150, 9
    kp, vp, pt = ref.make_cache(g, lens, hkv, 16)
    cu, seqs, at = _pack(rows, lens)
    q = _q(g, cu[-1], hq, dtype)
    for t, d in ((470, 3), (600, 9), (700, 70), (890, 100), (4, 120)):
        vp[int(pt[0, t // 16]), :, t % 16, d] = what
    out = api.attn_prompt_window(q, kp, vp, pt, _ints(cu), _ints(lens), SCALE, window, sinks)
    p = torch.tensor(at, device=DEV)
    hit = torch.isnan(out) if math.isnan(what) else out == what
    for t, d in ((470, 3), (600, 9), (700, 70), (890, 100)):
        assert bool((hit[:, :, d] == ((p >= t) & (p < t + window))[:, None]).all()), t
    assert bool(hit[:, :, 120].all())
    rest = [d for d in range(D) if d not in (3, 9, 70, 100, 120)]
    assert bool(torch.isfinite(out[:, :, rest]).all())
    clean = vp.clone()
    clean[~torch.isfinite(clean)] = 0
    want = api.attn_prompt_window(q, kp, clean, pt, _ints(cu), _ints(lens), SCALE, window, sinks)
    assert bool((out[:, :, rest] == want[:, :, rest]).all())


def test_prompt_windows_of_a_long_prompt(cuda_lib):
    g, r = _gen(9), np.random.default_rng(9)
    kp, vp, pt = ref.make_cache(g, [6000], 2, 16)
    for dtype, window, sinks in ((torch.bfloat16, 1000, 4), (torch.float32, 333, 200), (torch.bfloat16, 100000, 0)):
        q = _q(g, 6000, 8, dtype)
        out = api.attn_prompt_window(q, kp, vp, pt, _ints([0, 6000]), _ints([6000]), SCALE, window, sinks)
        _check_prompt(out, q, kp, vp, pt, [6000], [0] * 6000, list(range(6000)), window, sinks,
                      rows=r.choice(6000, 50, replace=False).tolist())
    assert api.check_device_error() == 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_prompt_scales_strides_and_rows_outside(cuda_lib, dtype):
    g = _gen(5)
    rows, lens, hq, hkv = [10, 50], [130, 50], 8, 2
    kp, vp, pt = ref.make_cache(g, lens, hkv, 16)
    qkv = _q(g, 70, hq + 2 * hkv, dtype)
    qkv[:4] = math.nan
    qkv[64:] = math.nan
    cu, seqs, at = _pack(rows, lens)
    for scale in (SCALE, -SCALE, 0.0):
        out = torch.full((70, hq, D), 7.0, dtype=dtype, device=DEV)
        api.attn_prompt_window(qkv[:, :hq], kp, vp, pt, _ints([c + 4 for c in cu]), _ints(lens), scale, 30, 2, out=out)
        _check_prompt(out[4:64], qkv[4:64, :hq], kp, vp, pt, lens, seqs, at, 30, 2, scale)
        assert bool((out[:4] == 7).all()) and bool((out[64:] == 7).all())
    out.fill_(7.0)
    api.attn_prompt_window(qkv[:, :hq], kp, vp, pt, _ints([4, 14, 64]), _ints([pt.shape[1] * 16 + 1, 50]), SCALE, 30, 2, out=out)
    assert api.check_device_error() == POS and bool((out[:14] == 7).all())
    _check_prompt(out[14:64], qkv[14:64, :hq], kp, vp, pt[1:], lens[1:], [0] * 50, list(range(50)), 30, 2)
    api.attn_prompt_window(qkv[:, :hq], kp, vp, pt, _ints([4, 2, 64]), _ints(lens), SCALE, 30, 2, out=out)
    assert api.check_device_error() == POS


def test_prompt_in_a_graph_with_other_lengths(cuda_lib):
    g = _gen(14)
    kp, vp, pt = ref.make_cache(g, [1500, 1500], 2, 16)
    ws = torch.zeros(api.attn_prompt_workspace_bytes(), dtype=torch.uint8, device=DEV)
    cu, lens, q = _ints([0, 100, 300]), _ints([1500, 1500]), _q(g, 300, 8, torch.bfloat16)
    out = torch.empty_like(q)

    def call():
        api.attn_prompt_window(q, kp, vp, pt, cu, lens, SCALE, 180, 5, out=out, workspace=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for rows, ns in (([300, 0], [301, 1500]), ([1, 299], [1, 700]), ([150, 150], [1500, 149])):
        c, seqs, at = _pack(rows, ns)
        cu.copy_(_ints(c))
        lens.copy_(_ints(ns))
        graph.replay()
        _check_prompt(out, q, kp, vp, pt, ns, seqs, at, 180, 5, rows=range(0, 300, 7))
    assert api.check_device_error() == 0


# ------------------------------------------------------------------------------------- the weights of packed rows


def _check_weights(sums, before, q, kp, pt, rows, lens, cu, last, window, sinks, scale=SCALE, seqs=None):
    """Every key of the sequences: a sum of weights is off by what each is off by, and by 2^-23 of itself for every
    addition on the way (rows in tiles of 64 columns, tiles one after another: at most 64 + rows of them)."""
    sums, before, q = sums.double().cpu(), before.double().cpu(), q.double().cpu()
    hkv = kp.shape[1]
    for b, (n, m) in enumerate(zip(rows, lens)):
        if seqs is not None and b not in seqs:
            continue
        used = min(n, last) if last else n
        assert torch.equal(sums[b, :, m:], before[b, :, m:])
        if used == 0 or m == 0:
            assert torch.equal(sums[b], before[b])
            continue
        k = ref.tokens(kp, pt[b], m)
        total, tol = torch.zeros((hkv, m), dtype=torch.float64), torch.zeros((hkv, m), dtype=torch.float64)
        touched = torch.zeros(m, dtype=torch.bool)
        for j in range(n - used, n):
            see = ref.visible(m - n + j, m, window, sinks)
            _, w, _, dot = ref.attend(q[cu[b] + j], k, k, see, scale)
            total += w
            tol += w * (ref.weight_bound(dot, int(see.sum())) + (64 + used) * 2.0 ** -24)
            touched |= see
        assert torch.equal(sums[b, :, :m][:, ~touched], before[b, :, :m][:, ~touched]), b
        tol += 2.0 ** -23 * (before[b, :, :m] + total) + 1e-30
        err = (sums[b, :, :m] - before[b, :, :m] - total).abs()
        assert bool((err <= tol).all()), (b, n, m, float((err / tol).max()))


WEIGHTS = [   # rows, lengths, q heads, kv heads, page size, last, window, first tokens
    ([1], [1], 4, 2, 16, 0, ALL, 0),
    ([1, 1, 1], [1, 17, 300], 8, 8, 16, 0, ALL, 0),
    ([128], [128], 4, 4, 16, 0, ALL, 0),
    ([129, 0, 127], [129, 40, 127], 4, 2, 32, 0, 64, 3),
    ([64, 65, 3, 31], [64, 65, 1000, 331], 32, 8, 16, 16, ALL, 0),
    ([300, 17], [300, 900], 16, 2, 64, 0, 200, 5),
    ([33, 70], [729, 470], 4, 2, 7, 20, 128, 128),
    ([40, 200], [40, 1500], 8, 2, 24, 33, ALL, 0),
    ([16, 20], [5, 20], 4, 2, 16, 0, ALL, 0),          # rows before position 0 see nothing
    ([9, 4], [0, 0], 4, 1, 16, 0, ALL, 0),
    ([1], [5000], 8, 1, 128, 0, ALL, 0),
    ([600], [900], 8, 2, 256, 0, ALL, 0),
    ([2, 0, 0, 1], [2, 0, 7, 257], 2, 2, 1, 0, 33, 2),
    ([500], [500], 2, 2, 16, 0, ALL, 0),
    ([260], [2500], 8, 1, 16, 40, 311, 213),
    ([2201], [2201], 8, 2, 16, 0, ALL, 0),
    ([32] * 9, [1800] * 9, 16, 4, 16, 32, ALL, 0),
    ([700, 40], [700, 90], 16, 2, 16, 0, 300, 0),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,lens,hq,hkv,ps,last,window,sinks", WEIGHTS)
def test_weights(cuda_lib, rows, lens, hq, hkv, ps, last, window, sinks, dtype):
    g = _gen(sum(rows) + hq)
    kp, vp, pt = ref.make_cache(g, lens, hkv, ps)
    cu, _, _ = _pack(rows, lens)
    q = _q(g, cu[-1], hq, dtype)
    before = torch.rand((len(rows), hkv, pt.shape[1] * ps), generator=g, device=DEV) * 0.1
    ws = torch.full((api.attn_key_weights_workspace_bytes(len(rows), cu[-1], hq, hkv, last),), 255, dtype=torch.uint8, device=DEV)
    ws[:16384] = 0      # what has to be
    got = []
    for _ in range(2):
        sums = before.clone()
        assert api.attn_key_weights(q, kp, pt, _ints(cu), _ints(lens), SCALE, sums, last, window, sinks, workspace=ws) is sums
        got.append(sums)
    assert torch.equal(*got)
    _check_weights(got[0], before, q, kp, pt, rows, lens, cu, last, window, sinks)
    assert api.check_device_error() == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("seed", range(6))
def test_weights_ragged(cuda_lib, seed, dtype):
    g, r = _gen(80 + seed), np.random.default_rng(seed)
    hq, hkv = [(8, 1), (4, 4), (32, 8), (16, 2), (8, 8), (16, 8)][seed]
    n = int(r.integers(1, 30))
    lens = [int(x) for x in 2 ** r.uniform(0, 11, n)]
    rows = [min(m, int(x)) for m, x in zip(lens, 2 ** r.uniform(0, 8, n))]
    window, sinks, ps = [ALL, int(2 ** r.uniform(0, 10))][seed % 2], int(r.integers(0, 300)), int(r.choice([7, 16, 24, 128]))
    last = [0, int(r.integers(1, 60))][seed // 2 % 2]
    kp, vp, pt = ref.make_cache(g, lens, hkv, ps)
    cu, _, _ = _pack(rows, lens)
    q = _q(g, cu[-1], hq, dtype, 1 + 4 * (seed % 3))
    sums = torch.zeros((n, hkv, pt.shape[1] * ps), device=DEV)
    before = sums.clone()
    api.attn_key_weights(q, kp, pt, _ints(cu), _ints(lens), SCALE, sums, last, window, sinks)
    _check_weights(sums, before, q, kp, pt, rows, lens, cu, last, window, sinks,
                   seqs=set(r.choice(n, min(n, 6), replace=False).tolist()))
    assert api.check_device_error() == 0


def test_weights_of_single_rows_are_the_decode_calls(cuda_lib):
    g = _gen(15)
    lens = [1, 700, 64, 2100]
    kp, vp, pt = ref.make_cache(g, lens, 2, 16)
    q = _q(g, 4, 8, torch.float32)
    a, b = (torch.zeros((4, 2, pt.shape[1] * 16), device=DEV) for _ in range(2))
    api.attn_key_weights(q, kp, pt, _ints([0, 1, 2, 3, 4]), _ints(lens), SCALE, a, window=500, n_sinks=3)
    api.attn_decode_window(q, kp, vp, pt, _ints(lens), SCALE, 500, 3, key_weights=b)
    assert float((a - b).abs().max()) < 2.0 ** -16 and float((a - b).norm() / b.norm()) < 2.0 ** -18


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", DTYPES)
def test_weights_hidden_and_visible_values(cuda_lib, dtype, bad):
    g = _gen(16)
    rows, lens, window, sinks = [90, 20, 1], [1150, 445, 700], 200, 20
    kp, vp, pt = ref.make_cache(g, lens, 2, 16)
    cu, _, _ = _pack(rows, lens)
    q = _q(g, cu[-1], 8, dtype)
    ck, cpt = kp.clone(), pt.clone()
    _gone(pt, kp, vp, lens, [m - n for n, m in zip(rows, lens)], window, sinks, 16, bad, True)
    sums = torch.zeros((3, 2, pt.shape[1] * 16), device=DEV)
    before = sums.clone()
    api.attn_key_weights(q, kp, pt, _ints(cu), _ints(lens), SCALE, sums, window=window, n_sinks=sinks)
    _check_weights(sums, before, q, ck, cpt, rows, lens, cu, 0, window, sinks)
    assert api.check_device_error() == 0
    # one that rows 60 .. of sequence 0 (tokens 1120 ..) see, in one kv head
    kp[int(pt[0, 70]), 1, 0, 3] = math.nan
    sums.zero_()
    api.attn_key_weights(q, kp, pt, _ints(cu), _ints(lens), SCALE, sums, window=window, n_sinks=sinks)
    assert bool(sums[0, 0].isfinite().all()) and bool(sums[1:].isfinite().all())
    nan = sums[0, 1].isnan()
    assert bool(nan[:20].all()) and not bool(nan[20:921].any()) and bool(nan[921:1150].all()) and not bool(nan[1150:].any())


def test_weights_refused_lengths_and_rows_outside(cuda_lib):
    g = _gen(17)
    rows, lens = [10, 50], [130, 50]
    kp, vp, pt = ref.make_cache(g, lens, 2, 16)
    qkv = _q(g, 70, 12, torch.bfloat16)
    qkv[:4] = math.nan
    qkv[64:] = math.nan
    sums = torch.zeros((2, 2, pt.shape[1] * 16), device=DEV)
    before = sums.clone()
    api.attn_key_weights(qkv[:, :8], kp, pt, _ints([4, 14, 64]), _ints(lens), -SCALE, sums)
    _check_weights(sums, before, qkv[4:, :8], kp, pt, rows, lens, [0, 10, 60], 0, ALL, 0, -SCALE)
    assert api.check_device_error() == 0
    sums.zero_()
    api.attn_key_weights(qkv[:, :8], kp, pt, _ints([4, 14, 64]), _ints([pt.shape[1] * 16 + 1, 50]), SCALE, sums)
    assert api.check_device_error() == POS and bool((sums[0] == 0).all())
    _check_weights(sums, before, qkv[4:, :8], kp, pt, rows, lens, [0, 10, 60], 0, ALL, 0, seqs={1})
    sums.zero_()
    api.attn_key_weights(qkv[:, :8], kp, pt, _ints([4, 2, 64]), _ints(lens), SCALE, sums)
    assert api.check_device_error() == POS and bool((sums == 0).all())
    assert bool((api.attn_key_weights(qkv[:0, :8], kp, pt, _ints([0, 0, 0]), _ints(lens), SCALE, sums) == 0).all())
    pt[1, 1] = -1
    api.attn_key_weights(qkv[:, :8], kp, pt, _ints([4, 14, 64]), _ints(lens), SCALE, sums)
    assert api.check_device_error() == PAGE


def test_numbers_past_32_bits_are_refused(cuda_lib):
    g = _gen(19)
    kp, vp, pt = ref.make_cache(g, [20], 2, 16)
    q, cu, n = _q(g, 1, 8, torch.float32), _ints([0, 1]), _ints([20])
    sums = torch.zeros((1, 2, 32), device=DEV)
    for bad in (2 ** 32 + 5, -2 ** 31 - 7):
        for kw in (dict(window=bad), dict(n_sinks=bad)):
            with pytest.raises(ValueError, match=str(bad)):
                api.attn_decode_window(q, kp, vp, pt, n, SCALE, **kw)
            with pytest.raises(ValueError, match=str(bad)):
                api.attn_prompt_window(q, kp, vp, pt, cu, n, SCALE, **kw)
            with pytest.raises(ValueError, match=str(bad)):
                api.attn_key_weights(q, kp, pt, cu, n, SCALE, sums, **kw)
        with pytest.raises(ValueError, match=str(bad)):
            api.attn_key_weights(q, kp, pt, cu, n, SCALE, sums, last=bad)
    for call in (lambda: api.attn_decode_window(q, kp, vp, pt, n, SCALE, 0),
                 lambda: api.attn_prompt_window(q, kp, vp, pt, cu, n, SCALE, 5, -1)):
        with pytest.raises(api.QDError, match="window="):
            call()


def test_weights_share_a_workspace_over_sizes_and_graphs(cuda_lib):
    # one workspace for calls of several sizes, captured and replayed in turn
    g = _gen(20)
    ws = torch.zeros(max(api.attn_key_weights_workspace_bytes(2, 900, 8, 2), api.attn_key_weights_workspace_bytes(1, 64, 16, 8)),
                     dtype=torch.uint8, device=DEV)
    runs = []
    for rows, lens, hq, hkv, dtype, last in (([700, 200], [700, 900], 8, 2, torch.float32, 0), ([64], [1500], 16, 8, torch.bfloat16, 16)):
        kp, vp, pt = ref.make_cache(g, lens, hkv, 16)
        cu, _, _ = _pack(rows, lens)
        q, cu_d, n = _q(g, cu[-1], hq, dtype), _ints(cu), _ints(lens)
        sums = torch.zeros((len(rows), hkv, pt.shape[1] * 16), device=DEV)

        def call(q=q, kp=kp, pt=pt, cu_d=cu_d, n=n, sums=sums, last=last):
            api.attn_key_weights(q, kp, pt, cu_d, n, SCALE, sums, last=last, workspace=ws)

        call()
        torch.cuda.synchronize()
        want = sums.clone()
        _check_weights(want, torch.zeros_like(want), q, kp, pt, rows, lens, cu, last, ALL, 0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        runs.append((graph, sums, want, call))     # (which holds the inputs)
    for _ in range(4):
        for graph, sums, want, _ in runs:
            sums.zero_()
            graph.replay()
            assert torch.equal(sums, want)
    assert bool((ws[:16384] == 0).all()) and api.check_device_error() == 0


def test_weights_in_a_graph_with_other_lengths(cuda_lib):
    g = _gen(18)
    kp, vp, pt = ref.make_cache(g, [600, 600], 2, 16)
    cu, lens, q = _ints([0, 100, 200]), _ints([600, 600]), _q(g, 200, 8, torch.float32)
    ws = torch.zeros(api.attn_key_weights_workspace_bytes(2, 200, 8, 2), dtype=torch.uint8, device=DEV)
    sums = torch.zeros((2, 2, pt.shape[1] * 16), device=DEV)

    def call():
        api.attn_key_weights(q, kp, pt, cu, lens, SCALE, sums, window=250, n_sinks=5, workspace=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for rows, ns in (([200, 0], [301, 600]), ([1, 199], [1, 400]), ([90, 110], [600, 109])):
        c, _, _ = _pack(rows, ns)
        cu.copy_(_ints(c))
        lens.copy_(_ints(ns))
        sums.zero_()
        graph.replay()
        _check_weights(sums, torch.zeros_like(sums), q, kp, pt, rows, ns, c, 0, 250, 5)
    assert api.check_device_error() == 0
