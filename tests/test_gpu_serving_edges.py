"""The serving operators at the edges of what their arguments allow: values that are not finite, starts and
sizes near 32 bits, broken page tables, borders that rounding could misplace."""
import math

import numpy as np
import pytest
import torch

import serving_reference as ref
from test_gpu_serving import D, DEV, SCALE, _cache, _check_rows, _gen, _ints, _pack
from transformer_decode_step_weight_gb300 import api

pytestmark = pytest.mark.gpu
LOW, HIGH = -2 ** 31, 2 ** 31 - 1


# starts whose differences pass 32 bits
@pytest.mark.parametrize("cu", [[2000000000, -2000000000], [5, LOW], [HIGH, LOW], [LOW, HIGH], [1, LOW + 3],
                                [0, HIGH, -5], [HIGH, LOW, 20], [0, 2000000000, -2000000000]])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_attention_starts_far_apart_are_refused(cuda_lib, monkeypatch, cu, dtype):
    monkeypatch.setenv("QD_SHARED_MIN_MB", "0")
    g = _gen(50)
    n = len(cu) - 1
    kp, vp, pt = _cache(g, [64] * n, 2, 16)
    q = torch.randn((20, 4, D), generator=g, device=DEV).to(dtype)
    out = torch.full_like(q, 3)
    api.attn_prompt(q, kp, vp, pt, _ints(cu), _ints([64] * n), SCALE, out=out)
    assert api.check_device_error() == 2 and bool((out == 3).all())
    pt20 = pt[:1].expand(20, -1).contiguous()
    api.attn_decode_shared(q, kp, vp, pt20, _ints([64] * 20), _ints(cu), _ints([32] * n), SCALE, out=out)
    assert api.check_device_error() == 2 and bool((out == 3).all())


@pytest.mark.parametrize("max_seqs,max_pages,new", [(2048, 1 << 20, 1 << 20), (1, 1 << 30, 1 << 30),
                                                    (2, 1 << 30, 1 << 30), (2048, 1 << 19, 1 << 19)])
def test_extension_by_more_pages_than_32_bits_count_is_refused_whole(cuda_lib, max_seqs, max_pages, new):
    # pages of one token: 2^31, 2^30, 2^31 and 2^30 of them are wanted, 64 exist
    g = _gen(51)
    k = [torch.randn((64, 1, 1, 8), generator=g, device=DEV).to(torch.bfloat16)]
    c = api.PageCache.empty(k, [k[0].clone()], max_seqs, max_pages)
    c.extend(_ints([5] + [0] * (max_seqs - 1)))
    before = c.refs.clone()
    c.extend(_ints([new - 5] + [new] * (max_seqs - 1)))
    assert api.check_device_error() == 32
    assert torch.equal(c.refs, before) and int(c.seq_lens.sum()) == 5
    assert c.page_table[0, :6].tolist() == [0, 1, 2, 3, 4, -1]
    for s in range(0, max_seqs, 97):
        assert bool((c.page_table[s, 5 if s == 0 else 0:] == -1).all())
    c.extend(_ints([59] + [0] * (max_seqs - 1)))     # the workspace is left ready
    assert api.check_device_error() == 0 and int(c.refs.sum()) == 64


def _steep(g, n, hq, hkv, ps, top, prompt_rows=1):
    """Caches of one sequence of n keys whose key `top` outweighs every other by far more than 32 bits hold."""
    kp, vp, pt = _cache(g, [n], hkv, ps)
    at = (pt[0, top // ps].long(), slice(None), top % ps)
    kp[at] = 30.0
    return kp, vp, pt


def _is_value(got, want):
    """A softmax of one weight w gives w v / w. f32: w v is the sum of three exact products (their adder truncates,
    3 x 2^-23 at most), w in three parts (2^-25), the reciprocal and two products round (3 x 2^-24), together below
    2^-20 of v. bf16: the weight's distance from 1 (a score of 490 rounded in f32, 2^-15) is below half a step of v,
    a bf16 value, so v comes back."""
    want = want.expand_as(got)
    off = (got.double() - want.double()).abs()
    assert bool((off <= (0 if got.dtype == torch.bfloat16 else 2.0 ** -20) * want.double().abs()).all())


def _put(pages, pt, ps, key, value, dim=slice(None), row=0):
    pages[int(pt[row, key // ps]), :, key % ps, dim] = value


# a visible NaN or infinity whose weight is below what 32 bits hold, in a piece of its own: before and after the
# piece that has all the weight
@pytest.mark.parametrize("top,low", [(4990, 10), (10, 4990), (2500, 300)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompt_attention_joins_what_is_not_finite_in_pieces_of_no_weight(cuda_lib, top, low, dtype):
    g = _gen(52)
    n, hq, hkv, ps = 5000, 8, 1, 16
    kp, vp, pt = _steep(g, n, hq, hkv, ps, top)
    q = torch.ones((1, hq, D), dtype=dtype, device=DEV)
    args = (q, kp, vp, pt, _ints([0, 1]), _ints([n]), SCALE)
    _put(vp, pt, ps, low, math.nan, 3)
    _put(vp, pt, ps, low, math.inf, 9)
    _put(vp, pt, ps, low, -math.inf, 100)
    out = api.attn_prompt(*args)[0]
    assert bool(torch.isnan(out[:, 3]).all())
    assert bool(torch.isposinf(out[:, 9]).all()) and bool(torch.isneginf(out[:, 100]).all())
    rest = [d for d in range(D) if d not in (3, 9, 100)]
    _is_value(out[:, rest], vp[int(pt[0, top // ps]), 0, top % ps][rest])   # one key has all the weight
    # a key of NaN: its weight is NaN, whatever the others'
    kp2, vp2, _ = _cache(g, [n], hkv, ps)
    _put(kp2, pt, ps, top, 30.0)
    _put(kp2, pt, ps, low, math.nan, 7)
    out = api.attn_prompt(q, kp2, vp2, pt, _ints([0, 1]), _ints([n]), SCALE)
    assert bool(torch.isnan(out).all())
    assert api.check_device_error() == 0


@pytest.mark.parametrize("top,low", [(2100, 10), (10, 3500), (3590, 2010), (2010, 3590), (50, 1990)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("min_mb", ["0", "80"])
def test_shared_attention_joins_nan_in_pieces_of_no_weight(cuda_lib, monkeypatch, top, low, dtype, min_mb):
    # keys of the prefix, of the own tokens' first split, of their last
    monkeypatch.setenv("QD_SHARED_MIN_MB", min_mb)
    g = _gen(53)
    hq, hkv, ps, shared, n = 8, 2, 16, 2000, 3600
    q = torch.ones((3, hq, D), dtype=dtype, device=DEV)
    for what in ("value", "key"):
        kp, vp, pt = _cache(g, [n] * 3, hkv, ps, [(0, shared // ps)] * 3)
        for row in range(3):
            _put(kp, pt, ps, top, 30.0, row=row)
            _put(vp if what == "value" else kp, pt, ps, low, math.nan, 3, row=row)
        out = api.attn_decode_shared(q, kp, vp, pt, _ints([n] * 3), _ints([0, 3]), _ints([shared]), SCALE)
        if what == "key":
            assert bool(torch.isnan(out).all())
            continue
        assert bool(torch.isnan(out[:, :, 3]).all())
        rest = [d for d in range(D) if d != 3]
        for row in range(3):
            want = vp[int(pt[row, top // ps]), :, top % ps].repeat_interleave(hq // hkv, 0)
            _is_value(out[row][:, rest], want[:, rest])
    assert api.check_device_error() == 0


# ---- scores of -inf (bf16 q; an f32 q splits into parts whose products with an infinity give NaN)


def _without(kp, vp, pt, row, n, gone):
    keep = [t for t in range(n) if t not in gone]
    return ref.gather(kp, pt[row], n)[keep], ref.gather(vp, pt[row], n)[keep]


def _near(got, q, k, v):
    out, mag, vmax, dot = ref.attend(q.double().cpu(), k, v, k.shape[0], SCALE)
    err = (got.double().cpu() - out).abs()
    assert bool((err <= ref.attention_bound(out, mag, vmax, dot, k.shape[0], True)).all()), float(err.max())


@pytest.mark.parametrize("gone", [[256], [0], [255, 256], [64, 65, 66], list(range(16)), list(range(0, 257, 2)),
                                  list(range(256))])
def test_scores_of_minus_infinity_weigh_nothing(cuda_lib, monkeypatch, gone):
    # whole blocks and warps whose only scores are -inf beside others that are finite
    g = _gen(54)
    n, hq, hkv, ps = 257, 8, 2, 16
    kp, vp, pt = _cache(g, [n], hkv, ps)
    for t in gone:
        _put(kp, pt, ps, t, -math.inf, 5)
    q = torch.randn((1, hq, D), generator=g, device=DEV).to(torch.bfloat16)
    q[:, :, 5] = 0.5
    k, v = _without(kp, vp, pt, 0, n, gone)
    _near(api.attn_prompt(q, kp, vp, pt, _ints([0, 1]), _ints([n]), SCALE)[0], q[0], k, v)
    pt2 = pt.expand(2, -1).contiguous()
    q2 = q.expand(2, -1, -1).contiguous()
    for min_mb in ("0", "80"):
        monkeypatch.setenv("QD_SHARED_MIN_MB", min_mb)
        for shared in (0, 100, 256, 257):
            out = api.attn_decode_shared(q2, kp, vp, pt2, _ints([n, n]), _ints([0, 2]), _ints([shared]), SCALE)
            for row in range(2):
                _near(out[row], q[0], k, v)
    assert api.check_device_error() == 0


@pytest.mark.parametrize("n", [1, 40, 300, 3000])
def test_rows_whose_scores_are_all_minus_infinity_are_nan(cuda_lib, monkeypatch, n):
    # keys are seen, so this is not the row of zeros that sees none: a sum of weights of 0 / 0
    g = _gen(55)
    hq, hkv, ps = 8, 2, 16
    kp, vp, pt = _cache(g, [n], hkv, ps)
    kp[:, :, :, 5] = -math.inf
    q = torch.randn((2, hq, D), generator=g, device=DEV).to(torch.bfloat16)
    q[:, :, 5] = 0.5
    out = api.attn_prompt(q, kp, vp, pt, _ints([0, 2]), _ints([n]), SCALE)
    assert bool(torch.isnan(out[1]).all())
    assert bool((out[0] == 0).all()) if n == 1 else bool(torch.isnan(out[0]).all())
    pt2 = pt.expand(2, -1).contiguous()
    for min_mb in ("0", "80"):
        monkeypatch.setenv("QD_SHARED_MIN_MB", min_mb)
        for shared in (0, n // 2, n):
            out = api.attn_decode_shared(q, kp, vp, pt2, _ints([n, 0]), _ints([0, 2]), _ints([shared]), SCALE)
            assert bool(torch.isnan(out[0]).all()) and bool((out[1] == 0).all())
    assert api.check_device_error() == 0


# ---- values that are not finite, seen by some rows or by all


@pytest.mark.parametrize("ps", [16, 24])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompt_attention_values_not_finite_reach_the_rows_that_see_them(cuda_lib, dtype, ps):
    # in both halves of the dims, in tiles that only some rows of a row tile see and in tiles that all see
    g = _gen(56)
    n, hq, hkv = 200, 8, 2
    kp, vp, pt = _cache(g, [n], hkv, ps)
    cu, seqs, seen = _pack([140], [n])
    q = torch.randn((140, hq, D), generator=g, device=DEV).to(dtype)
    clean = vp.clone()
    for key, value, dim in ((170, math.inf, 3), (180, -math.inf, 100), (150, math.nan, 64), (65, math.inf, 127),
                            (75, -math.inf, 127), (70, -math.inf, 0)):
        _put(vp, pt, ps, key, value, dim)
        _put(clean, pt, ps, key, 0.0, dim)
    out = api.attn_prompt(q, kp, vp, pt, _ints(cu), _ints([n]), SCALE)
    at = torch.tensor(seen, device=DEV)[:, None]
    assert bool((torch.isposinf(out[:, :, 3]) == (at > 170)).all())
    assert bool((torch.isneginf(out[:, :, 100]) == (at > 180)).all())
    assert bool((torch.isnan(out[:, :, 64]) == (at > 150)).all())
    assert bool((torch.isposinf(out[:, :, 127]) == ((at > 65) & (at <= 75))).all())
    assert bool((torch.isnan(out[:, :, 127]) == (at > 75)).all())
    assert bool((torch.isneginf(out[:, :, 0]) == (at > 70)).all())
    rest = [d for d in range(D) if d not in (0, 3, 64, 100, 127)]
    assert bool(torch.isfinite(out[:, :, rest]).all())
    # what is finite is right: the row's sum without the entries
    fixed = torch.where(torch.isfinite(out), out, 0)
    want = api.attn_prompt(q, kp, clean, pt, _ints(cu), _ints([n]), SCALE)
    _check_rows(torch.where(torch.isfinite(out), out, want), q, kp, clean, pt, seqs, seen, range(0, 140, 9))
    assert bool(torch.equal(fixed[:, :, rest], want[:, :, rest]))
    assert api.check_device_error() == 0


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompt_attention_values_not_finite_in_pieces(cuda_lib, dtype, rows):
    # a long cache in pieces: each patches its own keys
    g = _gen(57)
    n, hq, hkv, ps = 9000, 8, 2, 16
    kp, vp, pt = _cache(g, [n], hkv, ps)
    cu, seqs, seen = _pack([rows], [n])
    q = torch.randn((rows, hq, D), generator=g, device=DEV).to(dtype)
    clean = vp.clone()
    bad = ((100, math.inf, 3), (8998, -math.inf, 100), (4000, math.nan, 64), (20, math.inf, 127), (7000, -math.inf, 127),
           (8999, math.nan, 1))
    for key, value, dim in bad:
        _put(vp, pt, ps, key, value, dim)
        _put(clean, pt, ps, key, 0.0, dim)
    out = api.attn_prompt(q, kp, vp, pt, _ints(cu), _ints([n]), SCALE)
    want = api.attn_prompt(q, kp, clean, pt, _ints(cu), _ints([n]), SCALE)
    for r in range(rows):
        for dim, value in ((3, math.inf), (100, -math.inf if seen[r] > 8998 else None), (64, math.nan), (127, math.nan),
                           (1, math.nan if seen[r] > 8999 else None)):
            if value is None:
                continue
            got = out[r, :, dim]
            assert bool(torch.isnan(got).all() if math.isnan(value) else (got == value).all()), (r, dim)
            out[r, :, dim] = want[r, :, dim]
    assert torch.equal(out, want)
    assert api.check_device_error() == 0


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_shared_attention_prefix_values_that_some_rows_see(cuda_lib, monkeypatch, dtype, bad):
    # a value between the lengths of two sequences of the group
    monkeypatch.setenv("QD_SHARED_MIN_MB", "0")
    g = _gen(58)
    ps, hq, hkv, shared = 16, 8, 2, 200
    lens = [250, 100, 200, 5, 151, 150]
    kp, vp, pt = _cache(g, [256] * 6, hkv, ps, [(0, 13)] * 6)
    q = torch.randn((6, hq, D), generator=g, device=DEV).to(dtype)
    args = (_ints(lens), _ints([0, 6]), _ints([shared]), SCALE)
    want = api.attn_decode_shared(q, kp, vp, pt, *args)
    for dim in (3, 100):
        _put(vp, pt, ps, 150, bad, dim)
    out = api.attn_decode_shared(q, kp, vp, pt, *args)
    see = torch.tensor([n > 150 for n in lens], device=DEV)
    assert not bool(torch.isfinite(out[see][:, :, [3, 100]]).any())
    if math.isnan(bad):
        assert bool(torch.isnan(out[see][:, :, [3, 100]]).all())
    out[see.nonzero()[:, 0][:, None], :, torch.tensor([3, 100], device=DEV)] = \
        want[see.nonzero()[:, 0][:, None], :, torch.tensor([3, 100], device=DEV)]
    # the other dims and rows to the last bit but for the zeroed entry's own products
    _check_rows(out, q, kp, torch.where(torch.isfinite(vp), vp, 0), pt, list(range(6)), lens, [1, 3, 5])
    assert torch.equal(out[~see], want[~see])
    rest = [d for d in range(D) if d not in (3, 100)]
    assert torch.equal(out[:, :, rest], want[:, :, rest])
    assert api.check_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompt_attention_infinity_in_a_cache_of_300000_keys(cuda_lib, dtype):
    # two row tiles per SM, each over all the keys, looked through for the infinity while other roles wait
    g = _gen(59)
    n, hq, hkv, ps = 300000, 8, 1, 128
    rows = 2 * 152 * 16
    kp, vp, pt = _cache(g, [n], hkv, ps)
    _put(vp, pt, ps, 0, math.inf, 3)
    _put(vp, pt, ps, n - rows // 2, -math.inf, 70)
    q = torch.randn((rows, hq, D), generator=g, device=DEV).to(dtype)
    cu, seqs, seen = _pack([rows], [n])
    out = api.attn_prompt(q, kp, vp, pt, _ints(cu), _ints([n]), SCALE)
    assert api.check_device_error() == 0
    assert bool(torch.isposinf(out[:, :, 3]).all())
    at = torch.tensor(seen, device=DEV)[:, None]
    assert bool((torch.isneginf(out[:, :, 70]) == (at > n - rows // 2)).all())
    rest = [d for d in range(D) if d not in (3, 70)]
    assert bool(torch.isfinite(out[:, :, rest]).all())
    clean = torch.where(torch.isfinite(vp), vp, 0)
    fixed = torch.where(torch.isfinite(out), out, api.attn_prompt(q, kp, clean, pt, _ints(cu), _ints([n]), SCALE))
    _check_rows(fixed, q, kp, clean, pt, seqs, seen, [0, rows // 2 + 1, rows - 1])


def test_prompt_attention_looking_for_an_infinity_takes_a_few_times_the_call(cuda_lib):
    # a warp's lanes share the search: 6 times the call without (each for its own row: 87)
    g = _gen(60)
    n, hq, hkv, ps = 8192, 32, 8, 64
    kp, vp, pt = _cache(g, [n], hkv, ps)
    q = torch.randn((n, hq, D), generator=g, device=DEV).to(torch.bfloat16)
    ws = torch.zeros(api.attn_prompt_workspace_bytes(), dtype=torch.uint8, device=DEV)
    out, cu, ln = torch.empty_like(q), _ints([0, n]), _ints([n])

    def best():
        times = []
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            api.attn_prompt(q, kp, vp, pt, cu, ln, SCALE, out=out, workspace=ws)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    clean = best()
    _put(vp, pt, ps, 0, math.inf, 5)
    assert best() < 25 * clean
    assert bool(torch.isposinf(out[:, :, 5]).all()) and api.check_device_error() == 0


# ---- sampled verification near a border


def _near_border(r, u, tok, off):
    """Token tok has mass, and the running sums around it hold u times the sum, but for `off` of the sum."""
    c = np.cumsum(r.astype(np.float64))
    border, slack = u * c[-1], off * c[-1]
    assert r[tok] > 0 and c[tok] > border - slack and c[tok] - r[tok] <= border + slack, (tok, border, c[tok], r[tok])


def _flat_stretch(seed, nudge):
    """Masses whose border lies on a stretch of tokens without any: half of the sum on each side of it, up to
    `nudge` 2^-53."""
    g = np.random.default_rng(seed)
    r = np.zeros((256, 4), np.float32)
    live = g.random(100) < 0.5
    live[0] = live[99] = False
    live[60:] = False
    n = int(live.sum())
    r[:100][live] = (g.random((n, 4)) * 2.0 ** g.uniform(-12, 0, (n, 1)) / 400).astype(np.float32)
    half = float(r.astype(np.float64).sum())
    big = np.float32(half)
    rest = half - float(big) + nudge * 2.0 ** -53
    if rest < 0:
        big = np.nextafter(big, np.float32(0))
        rest = half - float(big) + nudge * 2.0 ** -53
    r[200, 0], r[210, 0] = big, np.float32(rest)
    r[220, 0] = np.float32(max(0.0, rest - float(np.float32(rest))))
    return r.ravel()


def test_verify_sample_border_on_a_stretch_without_mass(cuda_lib):
    # sums added in different orders disagree there in their last bits
    rows = [_flat_stretch(seed, k) for seed in [296] + list(range(100)) for k in range(-4, 5)]
    p = torch.from_numpy(np.stack(rows)).to(DEV)[:, None]
    B = len(rows)
    tok, pos, step = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(3))
    out = torch.zeros((B, 2), dtype=torch.int32, device=DEV)
    api.verify_sample(p, None, None, torch.full((B, 1), 0.5, device=DEV), tok, pos, step, out)
    for b, t in enumerate(tok.tolist()):
        _near_border(rows[b], 0.5, t, 2.0 ** -43)
    assert api.check_device_error() == 0


@pytest.mark.parametrize("V", [151936, 4000])
def test_verify_sample_border_among_many_small_masses(cuda_lib, V):
    # two tokens of a half, thousands of 2^-27 between them, multiples of 2^-48 all (exact in float32); the border 2^-41
    # before or behind the running sum of a small one, in a batch so large that each sequence is one chunk (594 and 16
    # tokens to a thread). A right kernel: groups of 16 are off by 120 2^-49 of their sum, half of the total at most,
    # two of them count, 14 additions of pairs by 1.5 2^-48 each: below 2^-41 together
    B, half, delta = 640, 1 << 47, 1 << 7
    g = _gen(61)
    m = torch.randint(1 << 21, 1 << 22, (B, V), generator=g, device=DEV)
    m[:, 0], m[:, V - 2:] = half, 0
    c = m.cumsum(1)
    j = torch.randint(V * 3 // 5, V - 10, (B,), generator=g, device=DEV)
    sign = torch.where(torch.arange(B, device=DEV) % 2 == 0, 1, -1)
    rest = 2 * (c.gather(1, j[:, None])[:, 0] + sign * delta) - c[:, -1]
    m[:, V - 2], m[:, V - 1] = rest >> 24 << 24, rest & ((1 << 24) - 1)
    assert bool((rest >= half).all())
    p = (m.double() * 2.0 ** -48).float()
    assert torch.equal((p.double() * 2.0 ** 48).long(), m)
    tok, pos, step = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(3))
    out = torch.zeros((B, 2), dtype=torch.int32, device=DEV)
    api.verify_sample(p[:, None], None, None, torch.full((B, 1), 0.5, device=DEV), tok, pos, step, out)
    want = torch.where(sign > 0, j + 1, j).int()
    assert torch.equal(tok, want), int((tok != want).sum())
    assert api.check_device_error() == 0


@pytest.mark.parametrize("bad", [-1, 20, 2 ** 31 - 1, -2 ** 31])
def test_page_operations_pass_over_table_entries_that_name_no_page(cuda_lib, bad):
    # pages of 4: sequence 0 has 5 pages (0 .. 4), sequence 1 has 2 (5, 6); sequence 0's third entry is broken
    g = _gen(62)
    k = [torch.randn((20, 2, 4, 8), generator=g, device=DEV).to(torch.bfloat16)]
    c = api.PageCache.empty(k, [k[0].clone()], 5, 6)
    c.extend(_ints([18, 7, 0, 0, 0]))
    assert api.check_device_error() == 0
    c.page_table[0, 2] = bad
    c.refs[2] = 0
    c.fork(_ints([0, 1]), _ints([3, 4]))          # as it is, the rest shared
    assert api.check_device_error() == 1
    assert c.page_table[3].tolist() == [0, 1, bad, 3, 4, -1] and c.page_table[4].tolist() == [5, 6, -1, -1, -1, -1]
    assert c.seq_lens.tolist() == [18, 7, 0, 18, 7]
    assert c.refs.tolist() == [2, 2, 0, 2, 2, 2, 2] + [0] * 13
    c.trim(_ints([4, -1, -1, -1, 0]))             # dropped, the rest given back
    assert api.check_device_error() == 1
    assert c.page_table[0].tolist() == [0] + [-1] * 5 and c.seq_lens.tolist() == [4, 7, 0, 18, 0]
    assert c.refs.tolist() == [2, 1, 0, 1, 1, 1, 1] + [0] * 13
    live = c.compact()                            # left, the rest moved: 6 goes to 2
    assert api.check_device_error() == 1 and int(live) == 6
    assert c.page_table[3].tolist() == [0, 1, bad, 3, 4, -1] and c.page_table[1, :2].tolist() == [5, 2]
    state = [t.clone() for t in (c.page_table, c.seq_lens, c.refs)]
    c.page_table[3, 4] = bad                      # the partly filled last page: nothing is changed
    state[0][3, 4] = bad
    c.extend(_ints([1, 1, 0, 1, 0]))
    assert api.check_device_error() == 33
    assert all(torch.equal(a, b) for a, b in zip(state, (c.page_table, c.seq_lens, c.refs)))
    # with a length past the table beside it: both errors, whichever thread comes first
    c.extend(_ints([1, 20, 0, 1, 0]))
    assert api.check_device_error() == 33
    assert all(torch.equal(a, b) for a, b in zip(state, (c.page_table, c.seq_lens, c.refs)))


@pytest.mark.parametrize("min_mb", ["0", "80"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_workspaces_need_zeros_in_their_head_only(cuda_lib, monkeypatch, dtype, min_mb):
    monkeypatch.setenv("QD_SHARED_MIN_MB", min_mb)
    g = _gen(63)
    hq, hkv, ps = 8, 2, 16
    lens = [3000, 2500, 900, 0, 40]
    kp, vp, pt = _cache(g, lens, hkv, ps, [(0, 50)] * 3 + [(1, 0)] * 2)
    q = torch.randn((5, hq, D), generator=g, device=DEV).to(dtype)
    ones = _ints(list(range(6)))
    shared = (q, kp, vp, pt, _ints(lens), _ints([0, 3, 5]), _ints([800, 0]), SCALE)
    p, d = (torch.softmax(torch.randn((5, k, 20000), generator=g, device=DEV), -1) for k in (3, 2))
    draft = torch.randint(0, 20000, (5, 2), generator=g, device=DEV).int()
    u = torch.rand((5, 3), generator=g, device=DEV)

    def verify(ws):
        state = [torch.zeros(5, dtype=torch.int32, device=DEV) for _ in range(3)]
        out = torch.zeros((5, 8), dtype=torch.int32, device=DEV)
        return torch.cat([api.verify_sample(p, d, draft, u, *state, out, workspace=ws)[:, None], out], 1)

    for call, nbytes, head in (
            (lambda ws: api.attn_prompt(q, kp, vp, pt, ones, _ints(lens), SCALE, workspace=ws),
             api.attn_prompt_workspace_bytes(), 8192),
            (lambda ws: api.attn_decode_shared(*shared, workspace=ws), api.attn_shared_workspace_bytes(5, hq, hkv), 8192),
            (verify, api.verify_sample_workspace_bytes(5), 20)):
        want = call(torch.zeros(nbytes, dtype=torch.uint8, device=DEV))
        ws = torch.full((nbytes,), 255, dtype=torch.uint8, device=DEV)
        ws[:head] = 0
        for _ in range(3):
            assert torch.equal(call(ws), want)
            assert int(ws[:head].max()) == 0     # left ready
        assert torch.equal(call(None), want)
    assert api.check_device_error() == 0


# ---- calls that share a workspace, the largest sizes


def test_one_workspace_for_both_attentions_and_two_graphs(cuda_lib, monkeypatch):
    g = _gen(64)
    hq, hkv, ps = 8, 2, 16
    lens = [3000, 2500, 2900]
    kp, vp, pt = _cache(g, lens, hkv, ps, [(0, 150)] * 3)
    ln, ones, cu, sl = _ints(lens), _ints([0, 1, 2, 3]), _ints([0, 3]), _ints([2400])
    ws = torch.zeros(api.attn_shared_workspace_bytes(3, hq, hkv), dtype=torch.uint8, device=DEV)
    qs = [torch.randn((3, hq, D), generator=g, device=DEV).to(t) for t in (torch.float32, torch.bfloat16)]

    def prompt(q, **kw):
        return api.attn_prompt(q, kp, vp, pt, ones, ln, SCALE, **kw)

    def shared(q, **kw):
        return api.attn_decode_shared(q, kp, vp, pt, ln, cu, sl, SCALE, **kw)

    graphs, want, outs = [], [], []
    for min_mb in ("0", "80"):
        monkeypatch.setenv("QD_SHARED_MIN_MB", min_mb)
        for q in qs:
            for call in (prompt, shared):
                want.append(call(q))
                for _ in range(2):
                    assert torch.equal(call(q, workspace=ws), want[-1])
                outs.append(torch.zeros_like(q))
                graphs.append(torch.cuda.CUDAGraph())
                with torch.cuda.graph(graphs[-1]):
                    call(q, out=outs[-1], workspace=ws)
    r = np.random.default_rng(64)
    for i in r.integers(0, len(graphs), 40):
        outs[i].zero_()
        graphs[i].replay()
        assert torch.equal(outs[i], want[i])
    assert api.check_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_attention_of_the_most_rows_and_sequences(cuda_lib, monkeypatch, dtype):
    g = _gen(65)
    n, B, ps = 1 << 20, 1024, 16
    kp, vp, _ = _cache(g, [1040], 1, ps, spare=0)
    pt = torch.randint(0, kp.shape[0], (B, 65), generator=g, device=DEV).int()
    lens = [1024 + b % 17 for b in range(B)]
    q = torch.randn((n, 1, D), generator=g, device=DEV).to(dtype)
    cu, seqs, seen = _pack([1024] * B, lens)
    out = api.attn_prompt(q, kp, vp, pt, _ints(cu), _ints(lens), SCALE)
    _check_rows(out, q, kp, vp, pt, seqs, seen, [0, 1023, 1024, 500000, 777777, n - 1024, n - 1])
    B = 65535
    pt = torch.randint(0, kp.shape[0], (B, 3), generator=g, device=DEV).int()
    starts = [min(B, 64 * i) for i in range(1025)]
    for i in range(0, 1024):
        pt[starts[i]:starts[i + 1], 0] = pt[starts[i], 0]
    lens = [16 + b % 33 for b in range(B)]
    for min_mb in ("0", "80"):
        monkeypatch.setenv("QD_SHARED_MIN_MB", min_mb)
        out = api.attn_decode_shared(q[:B], kp, vp, pt, _ints(lens), _ints(starts), _ints([16] * 1024), SCALE)
        _check_rows(out, q[:B], kp, vp, pt, list(range(B)), lens, [0, 63, 64, 30000, 65472, B - 1])
    assert api.check_device_error() == 0
