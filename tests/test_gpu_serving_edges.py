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
