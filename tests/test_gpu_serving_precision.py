"""The precision of the f32 attention: q and the softmax weights in three bf16 parts, O of each tile summed apart. Each
test has inputs whose exact result leaves one of these alone to matter, a bound derived from the arithmetic, and the
mistake it is there for planted in the oracle, which has to be out of the bound."""
import numpy as np
import pytest
import torch

from test_gpu_serving import D, DEV, _gen, _ints
from transformer_decode_step_weight_gb300 import api

pytestmark = pytest.mark.gpu
FORMS = ["prompt", "prefix", "own"]


def _attend(form, monkeypatch, q, kp, vp, n, scale):
    """q [B, Hq, D], every row over the same n keys, through one of the three kernels' paths."""
    monkeypatch.setenv("QD_SHARED_MIN_MB", "0" if form == "prefix" else "80")
    B = q.shape[0]
    row = torch.arange(kp.shape[0], dtype=torch.int32, device=DEV)
    if form == "prompt":
        assert B <= 1024
        pt = row.expand(B, -1).contiguous()
        return api.attn_prompt(q, kp, vp, pt, _ints(list(range(B + 1))), _ints([n] * B), scale)
    pt = row.expand(B, -1).contiguous()
    return api.attn_decode_shared(q, kp, vp, pt, _ints([n] * B), _ints([0, B]), _ints([n if form == "prefix" else 0]), scale)


def _parts(x, n):
    """The float32 value that n bf16 parts hold of x."""
    got = torch.zeros_like(x)
    for _ in range(n):
        got = got + (x - got).to(torch.bfloat16).float()
    return got


def _two_keys(size, ps=16):
    """Two keys, each with one entry of K (`size`) and one of V (1): the score of key i is size q[i], its weight O[i]."""
    kp = torch.zeros((1, 1, ps, D), dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros_like(kp)
    for i in range(2):
        kp[0, 0, i, i], vp[0, 0, i, i] = size, 1.0
    return kp, vp


def _softmax2(s):
    return torch.softmax(s.double(), -1)


@pytest.mark.parametrize("form", FORMS)
def test_f32_queries_enter_in_three_parts(cuda_lib, monkeypatch, form):
    # scores of about 96, as sums of the parts' products with 64: each is off by 2^-24 of itself (what three parts
    # leave) and two steps of the products' adder (2^-17 each), its scaling (own tokens) by half a step of 138 = 2^-17 in
    # log2 units; their difference by twice that and its own 2^-23; p moves by at most a quarter of it, and by 2^-19
    # through the weights and the division. Two parts leave up to 2^-16 of q
    g = _gen(70)
    B = 512
    kp, vp = _two_keys(64.0)
    q = torch.zeros((B, 1, D), device=DEV)
    q[:, 0, 0] = 1.5 + 0.05 * torch.rand(B, generator=g, device=DEV)
    q[:, 0, 1] = q[:, 0, 0] + 0.02 * (torch.rand(B, generator=g, device=DEV) - 0.5)
    bound = 0.25 * (2 * (100 * 2.0 ** -24 + 2 * 2.0 ** -17 + 0.7 * 2.0 ** -17) + 2.0 ** -23) + 2.0 ** -19
    want = _softmax2(64 * q[:, 0, :2].double())
    planted = (_softmax2(64 * _parts(q[:, 0, :2], 2).double()) - want).abs().max()
    assert float(planted) > 2 * bound
    out = _attend(form, monkeypatch, q, kp, vp, 2, 1.0)[:, 0]
    assert float((out[:, :2].double() - want).abs().max()) <= bound
    assert bool((out[:, 2:] == 0).all()) and api.check_device_error() == 0


@pytest.mark.parametrize("form", FORMS)
def test_f32_weights_enter_in_three_parts(cuda_lib, monkeypatch, form):
    # scores of at most 3: a difference of two is off by 2^-20 (two steps of the adder each), 2^-21.5 (their scaling) and
    # 6 2^-24; weights by 2^-22 each (the exponential), 2^-24 (three parts), their products' sums by two steps of 2^-23,
    # the sum, the reciprocal and the product by 2^-24 each: below 2^-18.4 of p. Two parts leave up to 2^-16 of a weight
    g = _gen(71)
    B = 1000
    kp, vp = _two_keys(1.0)
    q = torch.zeros((B, 1, D), device=DEV)
    q[:, 0, :2] = 6 * torch.rand((B, 2), generator=g, device=DEV) - 3
    bound = 2.0 ** -18.4
    s = q[:, 0, :2].double()
    want = _softmax2(s)
    w = torch.exp(s - s.max(-1, keepdim=True).values)
    planted = (_parts(w.float(), 2).double() / w.sum(-1, keepdim=True) / want - 1).abs().max()
    assert float(planted) > 2 * bound
    out = _attend(form, monkeypatch, q, kp, vp, 2, 1.0)[:, 0]
    assert float((out[:, :2].double() / want - 1).abs().max()) <= bound
    assert api.check_device_error() == 0


def _truncated_mean(v):
    """The mean of v [n] (float64 values of bf16) as sums of 16 added to one float32 that is cut off, not rounded."""
    total = np.float64(0)
    for part in v.reshape(-1, 16).sum(1):
        total += part
        near = np.float64(np.float32(total))
        total = np.float64(np.nextafter(np.float32(total), np.float32(0))) if near > total else near
    return total / len(v)


@pytest.mark.parametrize("form", ["prompt", "prefix"])
def test_f32_tiles_are_added_with_rounding(cuda_lib, monkeypatch, form):
    # every weight is 1 (K is 0), V in [2^-12, 2), a row tile of some 90 key tiles to each CTA. A tile's sum is made in 8
    # steps that cut off at most 2 2^-23 of what they have (half of it on average): 2^-20; some 94 tiles are added with
    # rounding, 47 2^-24; a row tile cut in up to three pieces, the reciprocal and the product: 8 2^-24. All of it in
    # one sum that is cut off loses some 2^-16
    g = _gen(72)
    n, ps, rows = 12032, 64, 152 * 16
    bound = 2.0 ** -20 + 55 * 2.0 ** -24
    kp = torch.zeros((n // ps, 1, ps, D), dtype=torch.bfloat16, device=DEV)
    vp = 1 + torch.rand((n // ps, 1, ps, D), generator=g, device=DEV)
    vp = (vp * 2.0 ** -torch.randint(0, 13, vp.shape, generator=g, device=DEV)).to(torch.bfloat16)
    q = torch.randn((rows, 8, D), generator=g, device=DEV)
    v = vp.double().reshape(n, D)
    if form == "prompt":
        row = torch.arange(n // ps, dtype=torch.int32, device=DEV)[None]
        out = api.attn_prompt(q, kp, vp, row, _ints([0, rows]), _ints([n]), 1.0)
        seen = torch.arange(n - rows + 1, n + 1, device=DEV)
        want = v.cumsum(0)[seen - 1] / seen[:, None]
    else:
        out = _attend(form, monkeypatch, q, kp, vp, n, 1.0)
        want = v.mean(0).expand(rows, -1)
    planted = max(abs(_truncated_mean(v[:, d].cpu().numpy()) / float(v[:, d].mean()) - 1) for d in range(4))
    assert planted > 2 * bound
    assert float((out.double() / want[:, None] - 1).abs().max()) <= bound
    assert api.check_device_error() == 0
