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
