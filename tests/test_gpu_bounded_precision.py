"""The precision of windowed attention and of key weights: an f32 q, and its softmax weights, in three bf16 parts, a
bf16 q's weights in two for single tokens. As in test_gpu_serving_precision.py the inputs leave one of these alone to
matter, and the mistake planted in the oracle is out of the bound."""
import pytest
import torch

from test_gpu_serving import D, DEV, _gen, _ints
from test_gpu_serving_precision import _parts, _softmax2, _two_keys
from transformer_decode_step_weight_gb300 import api

pytestmark = pytest.mark.gpu


def _attend(form, q, kp, vp):
    """q [B, 1, D], every row over both keys: O's first two values (form 'prompt', 'decode'), or the weights of the keys
    ('decode weights'; 'all rows': each walks the row tiles; 'last rows': each walks the keys)."""
    B = q.shape[0]
    pt, lens, cu = torch.zeros((B, 1), dtype=torch.int32, device=DEV), _ints([2] * B), _ints(list(range(B + 1)))
    sums = torch.zeros((B, 1, kp.shape[2]), device=DEV)
    if form == "prompt":
        out = api.attn_prompt_window(q, kp, vp, pt, cu, lens, 1.0, 2, 0)[:, 0]
    elif form.startswith("decode"):
        out = api.attn_decode_window(q, kp, vp, pt, lens, 1.0, 2, 0, key_weights=sums)[:, 0]
    else:
        api.attn_key_weights(q, kp, pt, cu, lens, 1.0, sums, last=int(form == "last rows"), window=2)
    if form in ("prompt", "decode"):
        assert bool((out[:, 2:] == 0).all())
        return out[:, :2].double()
    assert bool((sums[:, 0, 2:] == 0).all())
    return sums[:, 0, :2].double()


@pytest.mark.parametrize("form", ["prompt", "decode", "decode weights", "all rows", "last rows"])
def test_f32_queries_enter_in_three_parts(cuda_lib, form):
    # scores of about 96, as sums of the parts' products with 64: each is off by 2^-24 of itself (what three parts
    # leave), by two steps of the products' adder (2^-17 each; decode: one, and half a step where its two sums meet)
    # and by half a step of 138 = 2^-17 in log2 units (its scaling, or the reference maximum's); their difference by
    # twice that and its own 2^-23; p moves by at most a quarter of it, and by 2^-19 through the exponentials (2^-22
    # each), the parts, the sum and the division. Two parts leave up to 2^-16 of q
    g = _gen(170)
    B = 512
    kp, vp = _two_keys(64.0)
    q = torch.zeros((B, 1, D), device=DEV)
    q[:, 0, 0] = 1.5 + 0.05 * torch.rand(B, generator=g, device=DEV)
    q[:, 0, 1] = q[:, 0, 0] + 0.02 * (torch.rand(B, generator=g, device=DEV) - 0.5)
    bound = 0.25 * (2 * (100 * 2.0 ** -24 + 2 * 2.0 ** -17 + 0.7 * 2.0 ** -17) + 2.0 ** -23) + 2.0 ** -19
    want = _softmax2(64 * q[:, 0, :2].double())
    planted = (_softmax2(64 * _parts(q[:, 0, :2], 2).double()) - want).abs().max()
    assert float(planted) > 2 * bound
    assert float((_attend(form, q, kp, vp) - want).abs().max()) <= bound
    assert api.check_device_error() == 0


@pytest.mark.parametrize("form", ["prompt", "decode"])
def test_f32_weights_enter_in_three_parts(cuda_lib, form):
    # scores of at most 3: a difference of two is off by 2^-20 (two steps of the adder each), 2^-21.5 (their scaling) and
    # 6 2^-24; weights by 2^-22 each (the exponential), 2^-24 (three parts), their products' sums by two steps of 2^-23,
    # the sum, the reciprocal and the product by 2^-24 each: below 2^-18.4 of p. Two parts leave up to 2^-16 of a weight
    g = _gen(171)
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
    assert float((_attend(form, q, kp, vp) / want - 1).abs().max()) <= bound
    assert api.check_device_error() == 0


def test_bf16_decode_weights_enter_in_two_parts(cuda_lib):
    # values of 1 and -1 whose weights are nearly equal: the result is small, so its own rounding (2^-8 of it) is too,
    # and the weights' errors stand out: 2^-16 each (two parts), 2^-22 (the exponential), the scores' difference (of
    # exact bf16 scores around 2: two steps of 2^-22 and their scaling 2^-23 each) 2^-20, sums and division 2^-22.
    # One part leaves up to 2^-8 of a weight
    g = _gen(172)
    B = 1000
    kp, vp = _two_keys(1.0)
    vp.zero_()
    vp[0, 0, 0, 0], vp[0, 0, 1, 0] = 1.0, -1.0
    q = torch.zeros((B, 1, D), device=DEV)
    q[:, 0, 0] = 1 + torch.rand(B, generator=g, device=DEV)
    q[:, 0, 1] = q[:, 0, 0] + 0.06 * (torch.rand(B, generator=g, device=DEV) - 0.5)
    q = q.to(torch.bfloat16)
    s = q[:, 0, :2].double()
    p = _softmax2(s)
    want = p[:, 0] - p[:, 1]
    bound = 2.0 ** -16 + 2.0 ** -20 + 2.0 ** -21 + 2.0 ** -8 * want.abs()
    w = torch.exp(s - s.max(-1, keepdim=True).values)
    one = _parts(w.float(), 1).double()
    planted = ((one[:, 0] - one[:, 1]) / w.sum(-1) - want).abs()
    assert float((planted / bound).max()) > 2
    out = api.attn_decode_window(q, kp, vp, torch.zeros((B, 1), dtype=torch.int32, device=DEV), _ints([2] * B), 1.0, 2)
    assert bool(((out[:, 0, 0].double() - want).abs() <= bound).all())
    assert api.check_device_error() == 0
