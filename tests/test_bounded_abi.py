"""Refusals on the host of the operators that fill and bound the cache, before any CUDA call (no GPU)."""
import ctypes as C

import pytest
import torch

from transformer_decode_step_weight_gb300 import api, build

FAKE = 1 << 20     # never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.lib()


ROWS = dict(x=FAKE, f32=1, stride=48 * 128, qn=FAKE, kn=FAKE, eps=1e-6, cast=0, rope=FAKE, max_pos=100, pos=None,
            n_axes=1, axes=None, table=FAKE, cu=FAKE, lens=FAKE, batch=2, rows=10, hq=32, hkv=8, hd=128, ps=16,
            max_pages=4, n_pages=8, out=FAKE * 2, out_f32=1, k=FAKE, v=FAKE, stream=None)


@pytest.mark.parametrize("key,value,rc", [
    ("x", None, -1), ("qn", None, -1), ("kn", None, -1), ("rope", None, -1), ("table", None, -1), ("cu", None, -1),
    ("lens", None, -1), ("out", None, -1), ("k", None, -1), ("v", None, -1), ("x", FAKE + 8, -1), ("out", FAKE, -1),
    ("out", FAKE + 8, -1), ("rope", FAKE + 8, -1), ("qn", FAKE + 8, -1), ("f32", 2, -1), ("out_f32", -1, -1),
    ("cast", 2, -1), ("stride", 48 * 128 - 4, -1), ("stride", 48 * 128 + 2, -1), ("hd", 64, -2), ("eps", -1.0, -1),
    ("eps", float("nan"), -1), ("eps", float("inf"), -1), ("batch", 0, -1), ("batch", 1025, -2), ("rows", 0, -1),
    ("rows", (1 << 20) + 1, -2), ("hq", 0, -1), ("hkv", 1025, -2), ("ps", 0, -1), ("max_pages", 1 << 30, -1),
    ("max_pos", 0, -1), ("n_axes", 0, -1), ("n_axes", 5, -1), ("n_axes", 2, -1), ("axes", bytes([0] * 63 + [1]), -1)])
def test_rows_refusals(lib, key, value, rc):
    assert lib.qd_qk_norm_rope(*{**ROWS, key: value}.values()) == rc
    assert lib.qd_last_error().startswith(b"qd_qk_norm_rope: ")


def test_rows_binding_refuses():
    x, w = torch.zeros((2, 8 * 128)), torch.ones(128, dtype=torch.bfloat16)
    kv = torch.zeros((3, 2, 16, 128), dtype=torch.bfloat16)
    pt, n = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    rest = (w, w, torch.zeros((4, 64, 2)), kv, kv, pt, n, n, 1e-6)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        api.qk_norm_rope(x.half(), *rest)
    with pytest.raises(ValueError, match="contiguous"):
        api.qk_norm_rope(torch.zeros((8 * 128, 2)).T, *rest)
    with pytest.raises(ValueError, match="CUDA device"):
        api.qk_norm_rope(x, *rest)


DECODE = dict(q=FAKE, f32=0, stride=32 * 128, k=FAKE, v=FAKE, table=FAKE, lens=FAKE, batch=10, hq=32, hkv=8, hd=128,
              ps=16, max_pages=4, n_pages=8, scale=0.1, window=10, sinks=2, weights=FAKE, out=FAKE * 2, ws=FAKE,
              ws_bytes=1 << 40, stream=None)
ATTN_BAD = [("q", None, -1), ("out", None, -1), ("table", None, -1), ("lens", None, -1), ("ws", None, -1),
            ("k", FAKE + 8, -1), ("q", FAKE + 4, -1), ("out", FAKE, -1), ("f32", 2, -1), ("stride", 32 * 128 - 8, -1),
            ("stride", 32 * 128 + 4, -1), ("hd", 64, -2), ("hq", 12, -1), ("hq", 24, -2), ("ps", 0, -1),
            ("max_pages", 1 << 30, -1), ("scale", float("nan"), -1), ("ws_bytes", 0, -4), ("batch", 0, -1),
            ("n_pages", 1 << 26, -2), ("window", 0, -1), ("window", -5, -1), ("sinks", -1, -1)]


@pytest.mark.parametrize("key,value,rc", ATTN_BAD + [("batch", 65536, -2), ("weights", FAKE + 2, -1)])
def test_decode_refusals(lib, key, value, rc):
    assert lib.qd_attn_decode_window(*{**DECODE, key: value}.values()) == rc
    assert lib.qd_last_error().startswith(b"qd_attn_decode_window: ")


def test_decode_workspace(lib):
    n = api.attn_decode_window_workspace_bytes
    assert 0 == n(0, 8, 2) == n(1, 1, 2) == n(1, 8, 2, -1) and n(1, 8, 2) > 16384
    assert n(4, 32, 8, 1000) >= n(4, 32, 8) + 4 * 32 * 1000 * 4
    need = n(10, 32, 8, 12)
    assert lib.qd_attn_decode_window(*{**DECODE, "ws_bytes": need - 1}.values()) == -4
    assert lib.qd_attn_decode_window(*{**DECODE, "weights": None, "ws_bytes": n(10, 32, 8) - 1}.values()) == -4


PROMPT = dict(q=FAKE, f32=0, stride=32 * 128, k=FAKE, v=FAKE, table=FAKE, cu=FAKE, lens=FAKE, batch=2, rows=10, hq=32,
              hkv=8, hd=128, ps=16, max_pages=4, n_pages=8, scale=0.1, window=10, sinks=2, out=FAKE * 2, ws=FAKE,
              ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("key,value,rc", ATTN_BAD + [("cu", None, -1), ("batch", 1025, -2), ("rows", 0, -1),
                                                     ("rows", (1 << 20) + 1, -2)])
def test_prompt_refusals(lib, key, value, rc):
    assert lib.qd_attn_prompt_window(*{**PROMPT, key: value}.values()) == rc
    assert lib.qd_last_error().startswith(b"qd_attn_prompt_window: ")


WEIGHTS = dict(q=FAKE, f32=0, stride=32 * 128, k=FAKE, table=FAKE, cu=FAKE, lens=FAKE, batch=2, rows=10, hq=32, hkv=8,
               hd=128, ps=16, max_pages=4, n_pages=8, scale=0.1, last=0, window=10, sinks=2, weights=FAKE, ws=FAKE * 2,
               ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("key,value,rc", [b for b in ATTN_BAD if b[0] != "out"]
                         + [("cu", None, -1), ("batch", 1025, -2), ("rows", 0, -1), ("rows", (1 << 20) + 1, -2),
                            ("last", -1, -1), ("weights", None, -1), ("weights", FAKE + 2, -1), ("ws", FAKE + 8, -1)])
def test_weights_refusals(lib, key, value, rc):
    assert lib.qd_attn_key_weights(*{**WEIGHTS, key: value}.values()) == rc
    assert lib.qd_last_error().startswith(b"qd_attn_key_weights: ")


def test_weights_workspace(lib):
    n = api.attn_key_weights_workspace_bytes
    assert 0 == n(0, 5, 8, 2) == n(1, 0, 8, 2) == n(1, 5, 1, 2) == n(1, 5, 8, 2, -1)
    assert n(8, 8000, 32, 8, 32) < n(8, 8000, 32, 8)
    assert lib.qd_attn_key_weights(*{**WEIGHTS, "f32": 1, "ws_bytes": n(2, 10, 32, 8) - 1}.values()) == -4


def test_evict_refusals(lib):
    def cache(**kw):
        arr = (C.c_void_p * 2)(FAKE, FAKE)
        a = api.PageCacheArgs(C.cast(arr, C.c_void_p), C.cast(arr, C.c_void_p), 2, 8, 16, 128, 64, FAKE, FAKE, FAKE, 4, 8,
                              FAKE, 1 << 30)
        a.keep = arr
        for k, v in kw.items():
            setattr(a, k, v)
        return C.byref(a)

    def call(c, w=FAKE, keep=FAKE, sinks=0, recent=0):
        return lib.qd_pages_evict(c, w, keep, sinks, recent, None)

    assert call(None) == -1
    for kw, rc in ((dict(k_cache=None), -1), (dict(n_layers=0), -1), (dict(page_size=0), -1), (dict(head_dim=12), -2),
                   (dict(head_dim=264), -2), (dict(page_table=None), -1),
                   (dict(seq_lens=None), -1), (dict(refs=None), -1), (dict(workspace=None), -1), (dict(max_seqs=2049), -2),
                   (dict(max_pages=1 << 30), -1), (dict(workspace_bytes=16), -4)):
        c = cache(**kw)
        assert call(c) == rc, kw
    c = cache()
    assert call(c, w=None) == -1 and call(c, keep=None) == -1 and call(c, w=FAKE + 2) == -1
    assert call(c, sinks=-1) == -1 and call(c, recent=-1) == -1
    assert lib.qd_last_error().startswith(b"qd_pages_evict: ")
    assert call(cache(n_pages=1 << 26, workspace_bytes=1 << 40)) == -2
