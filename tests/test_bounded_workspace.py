"""Workspace of the key weights by q's type (no GPU)."""
import pytest
import torch

from test_bounded_abi import WEIGHTS
from transformer_decode_step_weight_gb300 import api, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.lib()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_call_takes_its_types_size(lib, dtype):
    need = api.attn_key_weights_workspace_bytes(2, 10, 32, 8, 0, dtype)
    f32 = int(dtype is torch.float32)
    assert need == lib.qd_attn_key_weights_workspace_bytes_for(f32, 2, 10, 32, 8, 0)
    assert lib.qd_attn_key_weights(*{**WEIGHTS, "f32": f32, "ws_bytes": need - 1}.values()) == -4
    assert str(need).encode() in lib.qd_last_error()      # what it asks for


def test_sizes(lib):
    n = api.attn_key_weights_workspace_bytes
    assert n(8, 8000, 32, 8) == lib.qd_attn_key_weights_workspace_bytes(8, 8000, 32, 8, 0)      # either type's
    tiles = (8000 * 4 // 128 + 8) * 8
    assert n(8, 8000, 32, 8) - n(8, 8000, 32, 8, dtype=torch.bfloat16) == tiles * 2 * 32768
    assert 0 == n(0, 5, 8, 2, 0, torch.bfloat16) == lib.qd_attn_key_weights_workspace_bytes_for(2, 1, 5, 8, 2, 0)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        n(1, 5, 8, 2, 0, torch.float16)
