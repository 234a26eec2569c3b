"""Refusals of the serving operators on the host, before any CUDA call, and the layout of
their struct (no GPU)."""
import ctypes as C
import os
import subprocess

import pytest
import torch

from transformer_decode_step_weight_gb300 import api, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20     # never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.lib()


def test_page_cache_struct_matches_c(tmp_path):
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "qd.h"\nint main(void) {\n'
                   '  printf("%zu %zu %zu %zu %zu\\n", sizeof(qd_page_cache), offsetof(qd_page_cache, n_pages),\n'
                   '         offsetof(qd_page_cache, refs), offsetof(qd_page_cache, max_pages),\n'
                   '         offsetof(qd_page_cache, workspace_bytes));\n  return 0;\n}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-I", "/usr/local/cuda/include", str(src), "-o",
                    str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    S = api.PageCacheArgs
    assert got == [C.sizeof(S), S.n_pages.offset, S.refs.offset, S.max_pages.offset, S.workspace_bytes.offset]


PROMPT = dict(q=FAKE, f32=0, stride=32 * 128, k=FAKE, v=FAKE, table=FAKE, cu=FAKE, lens=FAKE, batch=2, rows=10, hq=32,
              hkv=8, hd=128, ps=16, max_pages=4, n_pages=8, scale=0.1, out=FAKE * 2, ws=FAKE, ws_bytes=1 << 40, stream=None)
SHARED = dict(q=FAKE, f32=0, stride=32 * 128, k=FAKE, v=FAKE, table=FAKE, lens=FAKE, cu=FAKE, shared=FAKE, groups=2,
              batch=10, hq=32, hkv=8, hd=128, ps=16, max_pages=4, n_pages=8, scale=0.1, out=FAKE * 2, ws=FAKE,
              ws_bytes=1 << 40, stream=None)
ROWS_BAD = [("q", None, -1), ("out", None, -1), ("table", None, -1), ("lens", None, -1), ("cu", None, -1),
            ("ws", None, -1), ("k", FAKE + 8, -1), ("q", FAKE + 4, -1), ("out", FAKE, -1), ("f32", 2, -1),
            ("stride", 32 * 128 - 8, -1), ("stride", 32 * 128 + 4, -1), ("hd", 64, -2), ("hq", 12, -1), ("hq", 24, -2),
            ("ps", 0, -1), ("max_pages", 1 << 30, -1), ("scale", float("nan"), -1), ("scale", float("inf"), -1),
            ("ws_bytes", 0, -4), ("batch", 0, -1), ("n_pages", 1 << 26, -2)]


@pytest.mark.parametrize("key,value,rc", ROWS_BAD + [("batch", 1025, -2), ("rows", 0, -1), ("rows", (1 << 20) + 1, -2)])
def test_prompt_attention_refusals(lib, key, value, rc):
    assert lib.qd_attn_prompt(*{**PROMPT, key: value}.values()) == rc
    assert lib.qd_last_error().startswith(b"qd_attn_prompt: ")


@pytest.mark.parametrize("key,value,rc", ROWS_BAD + [("shared", None, -1), ("groups", 0, -1), ("groups", 1025, -2),
                                                     ("batch", 65536, -2)])
def test_shared_attention_refusals(lib, key, value, rc):
    assert lib.qd_attn_decode_shared(*{**SHARED, key: value}.values()) == rc
    assert lib.qd_last_error().startswith(b"qd_attn_decode_shared: ")


def _cache(**kw):
    arr = (C.c_void_p * 2)(FAKE, FAKE)
    a = api.PageCacheArgs(C.cast(arr, C.c_void_p), C.cast(arr, C.c_void_p), 2, 8, 16, 128, 64, FAKE, FAKE, FAKE, 4, 8,
                          FAKE, 1 << 30)
    a.keep = arr
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_page_operation_refusals(lib):
    calls = {"copy": lambda c: lib.qd_pages_copy(c, FAKE, FAKE, 1, None),
             "fork": lambda c: lib.qd_pages_fork(c, FAKE, FAKE, 1, None),
             "extend": lambda c: lib.qd_pages_extend(c, FAKE, None),
             "trim": lambda c: lib.qd_pages_trim(c, FAKE, None),
             "compact": lambda c: lib.qd_pages_compact(c, FAKE, None)}
    for name, call in calls.items():
        assert call(None) == -1
        assert call(C.byref(_cache(n_pages=0))) == -1, name
        if name in ("copy", "extend", "compact"):
            assert call(C.byref(_cache(k_cache=None))) == -1, name
            assert call(C.byref(_cache(n_layers=0))) == -1, name
            assert call(C.byref(_cache(page_size=0))) == -1, name
            assert call(C.byref(_cache(head_dim=12))) == -2, name
            bad = (C.c_void_p * 2)(FAKE, FAKE + 8)
            assert call(C.byref(_cache(v_cache=C.cast(bad, C.c_void_p)))) == -1, name
        if name != "copy":
            for k in ("page_table", "seq_lens", "refs", "workspace"):
                assert call(C.byref(_cache(**{k: None}))) == -1, (name, k)
            assert call(C.byref(_cache(max_seqs=0))) == -1, name
            assert call(C.byref(_cache(max_seqs=2049))) == -2, name
            assert call(C.byref(_cache(max_pages=1 << 30))) == -1, name
            assert call(C.byref(_cache(workspace_bytes=16))) == -4, name
    c = C.byref(_cache())
    assert lib.qd_pages_copy(c, None, FAKE, 1, None) == -1 and lib.qd_pages_copy(c, FAKE, FAKE, -1, None) == -1
    assert lib.qd_pages_fork(c, FAKE, None, 1, None) == -1 and lib.qd_pages_fork(c, FAKE, FAKE, 5, None) == -1
    assert lib.qd_pages_copy(c, None, None, 0, None) == 0 and lib.qd_pages_fork(c, None, None, 0, None) == 0
    assert lib.qd_pages_extend(c, None, None) == -1 and lib.qd_pages_trim(c, None, None) == -1
    assert lib.qd_pages_compact(c, None, None) == -1
    assert lib.qd_pages_workspace_bytes(None) == 0


VERIFY = dict(p=FAKE, ps=1000, q=FAKE, qs=1000, draft=FAKE, n_draft=None, u=FAKE, vocab=1000, batch=2, k=3, tok=FAKE,
              pos=FAKE, step=FAKE, out=FAKE, max_steps=8, m=FAKE, ws=FAKE, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("key,value,rc", [("p", None, -1), ("q", None, -1), ("draft", None, -1), ("u", None, -1),
                                          ("tok", None, -1), ("pos", None, -1), ("step", None, -1), ("out", None, -1),
                                          ("m", None, -1), ("ws", None, -1), ("ps", 999, -1), ("qs", 999, -1),
                                          ("vocab", 0, -1), ("batch", 0, -1), ("k", 0, -1), ("max_steps", 0, -1),
                                          ("vocab", 4194305, -2), ("batch", 65536, -2), ("k", 1025, -2),
                                          ("ws", FAKE + 4, -1), ("ws_bytes", 100, -4)])
def test_verify_sample_refusals(lib, key, value, rc):
    assert lib.qd_verify_sample(*{**VERIFY, key: value}.values()) == rc


def test_binding_refuses_host_tensors_and_wrong_shapes():
    q = torch.zeros((2, 4, 128))
    kv = torch.zeros((3, 2, 16, 128), dtype=torch.bfloat16)
    pt, n = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        api.attn_prompt(q, kv, kv, pt, torch.zeros(2, dtype=torch.int32), n, 0.1)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        api.attn_prompt(q.half(), kv, kv, pt, torch.zeros(2, dtype=torch.int32), n, 0.1)
    with pytest.raises(ValueError, match="contiguous"):
        api.attn_decode_shared(q.transpose(1, 2), kv, kv, pt, n, torch.zeros(2, dtype=torch.int32), n, 0.1)
    with pytest.raises(ValueError, match="CUDA device"):
        api.PageCache([kv], [kv])
    with pytest.raises(ValueError, match="V caches"):
        api.PageCache([kv], [])
    with pytest.raises(ValueError, match="float32"):
        api.verify_sample(q.half(), None, None, q, n, n, n, pt)
    with pytest.raises(ValueError, match="evenly spaced|CUDA"):
        api.verify_sample(torch.zeros((2, 3, 8)).transpose(0, 1), torch.zeros((3, 1, 8)), pt, q, n, n, n, pt)
