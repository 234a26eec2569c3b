"""Thin ctypes binding of libqd.so (argument marshalling only).

Every function here forwards device pointers (``tensor.data_ptr()``), sizes
and the current CUDA stream to the C ABI declared in ``include/qd.h``; all
arithmetic of the decode step runs in the library's CUDA kernels. PyTorch only
allocates device memory and supplies streams. If the library has not been
built, the first call raises: there is no fallback.
"""
from __future__ import annotations

import ctypes as C
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqd.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "qd.h")

QD_OK = 0
QD_W_BF16, QD_W_Q8_0, QD_W_INT4 = 0, 1, 2
QD_ACT_F32, QD_ACT_I8 = 0, 1
DEVERR = {1: "page", 2: "pos", 4: "nan", 8: "steps", 16: "timeout", 32: "cache"}

_vp = C.c_void_p
_i = C.c_int
_f = C.c_float
_sz = C.c_size_t
_l = C.c_int64


class LayerDims(C.Structure):
    _fields_ = [("hidden", _i), ("n_q_heads", _i), ("n_kv_heads", _i), ("head_dim", _i), ("ffn", _i),
                ("rms_eps", _f), ("rope_theta", _f), ("wtype", _i), ("act", _i)]


class LayerWeights(C.Structure):
    _fields_ = [(n, _vp) for n in ("w_qkv", "w_o", "w_gu", "w_down", "s_qkv", "s_o", "s_gu", "s_down",
                                   "ln_in", "ln_post", "q_norm", "k_norm")]


class StepArgs(C.Structure):
    _fields_ = [("layers", _vp), ("n_layers", _i),
                ("embed", _vp), ("final_norm", _vp), ("lm_head", _vp), ("lm_head_scales", _vp),
                ("lm_act", _i), ("vocab", _i),
                ("k_cache", _vp), ("v_cache", _vp),
                ("page_table", _vp), ("page_size", _i), ("max_pages", _i), ("n_pages", _i),
                ("rope_table", _vp), ("rope_max_pos", _i),
                ("tok", _vp), ("pos", _vp), ("step", _vp), ("out_tokens", _vp),
                ("max_steps", _i), ("batch", _i),
                ("logits", _vp), ("workspace", _vp), ("workspace_bytes", _sz),
                ("lm_wtype", _i), ("top_k", _i), ("topk_ids", _vp), ("topk_vals", _vp)]


class PageCacheArgs(C.Structure):
    _fields_ = [("k_cache", _vp), ("v_cache", _vp),
                ("n_layers", _i), ("n_kv_heads", _i), ("page_size", _i), ("head_dim", _i), ("n_pages", _i),
                ("page_table", _vp), ("seq_lens", _vp), ("refs", _vp), ("max_seqs", _i), ("max_pages", _i),
                ("workspace", _vp), ("workspace_bytes", _sz)]


_SIGS = {
    "qd_last_error": (C.c_char_p, []),
    "qd_version": (_i, []),
    "qd_gemv_bf16": (_i, [_vp, _i, _i, _vp, _i, _vp, _i, _vp]),
    "qd_gemv_q8_0": (_i, [_vp, _vp, _i, _i, _vp, _vp, _vp, _i, _vp, _vp]),
    "qd_quantize_q8_0": (_i, [_vp, _i, _vp, _vp, _vp]),
    "qd_gemv_w4": (_i, [_vp, _vp, _i, _i, _vp, _vp, _vp]),
    "qd_w4_topk_workspace_bytes": (_sz, []),
    "qd_gemv_w4_topk": (_i, [_vp, _vp, _i, _i, _vp, _i, _vp, _vp, _vp, _vp, _sz, _vp]),
    "qd_gemm_workspace_bytes": (_sz, [_i, _i, _i]),
    "qd_gemm_q8_0": (_i, [_vp, _vp, _i, _i, _vp, _i, _vp, _vp, _sz, _vp]),
    "qd_attn_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "qd_attn_decode_paged": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _vp, _vp, _sz, _vp]),
    "qd_attn_decode_paged_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _vp, _vp]),
    "qd_attn_prompt_workspace_bytes": (_sz, []),
    "qd_attn_prompt": (_i, [_vp, _i, _l] + [_vp] * 5 + [_i] * 8 + [_f, _vp, _vp, _sz, _vp]),
    "qd_attn_shared_workspace_bytes": (_sz, [_i, _i, _i]),
    "qd_attn_decode_shared": (_i, [_vp, _i, _l] + [_vp] * 6 + [_i] * 8 + [_f, _vp, _vp, _sz, _vp]),
    "qd_attn_prompt_window": (_i, [_vp, _i, _l] + [_vp] * 5 + [_i] * 8 + [_f, _i, _i, _vp, _vp, _sz, _vp]),
    "qd_attn_decode_window_workspace_bytes": (_sz, [_i, _i, _i, _l]),
    "qd_attn_decode_window": (_i, [_vp, _i, _l] + [_vp] * 4 + [_i] * 7 + [_f, _i, _i, _vp, _vp, _vp, _sz, _vp]),
    "qd_attn_key_weights_workspace_bytes": (_sz, [_i] * 5),
    "qd_attn_key_weights_workspace_bytes_for": (_sz, [_i] * 6),
    "qd_attn_key_weights": (_i, [_vp, _i, _l] + [_vp] * 4 + [_i] * 8 + [_f, _i, _i, _i, _vp, _vp, _sz, _vp]),
    "qd_qk_norm_rope": (_i, [_vp, _i, _l, _vp, _vp, _f, _i, _vp, _i, _vp, _i, C.c_char_p, _vp, _vp, _vp] + [_i] * 8
                        + [_vp, _i, _vp, _vp, _vp]),
    "qd_pages_workspace_bytes": (_sz, [C.POINTER(PageCacheArgs)]),
    "qd_pages_copy": (_i, [C.POINTER(PageCacheArgs), _vp, _vp, _i, _vp]),
    "qd_pages_fork": (_i, [C.POINTER(PageCacheArgs), _vp, _vp, _i, _vp]),
    "qd_pages_extend": (_i, [C.POINTER(PageCacheArgs), _vp, _vp]),
    "qd_pages_trim": (_i, [C.POINTER(PageCacheArgs), _vp, _vp]),
    "qd_pages_compact": (_i, [C.POINTER(PageCacheArgs), _vp, _vp]),
    "qd_pages_evict": (_i, [C.POINTER(PageCacheArgs), _vp, _vp, _i, _i, _vp]),
    "qd_verify_sample_workspace_bytes": (_sz, [_i]),
    "qd_verify_sample": (_i, [_vp, _l, _vp, _l, _vp, _vp, _vp, _i, _i, _i] + [_vp] * 4 + [_i, _vp, _vp, _sz, _vp]),
    "qd_argmax_workspace_bytes": (_sz, [_i]),
    "qd_argmax_advance": (_i, [_vp, _i, _i, _vp, _vp, _vp, _vp, _i, _vp, _sz, _vp]),
    "qd_rope_table_init": (_i, [_vp, _i, _i, _f, _vp]),
    "qd_create_layer": (_i, [C.POINTER(LayerDims), C.POINTER(LayerWeights), C.POINTER(_vp)]),
    "qd_destroy_layer": (_i, [_vp]),
    "qd_step_workspace_bytes": (_sz, [C.POINTER(StepArgs)]),
    "qd_decode_step": (_i, [C.POINTER(StepArgs), _vp]),
    "qd_step_launch_count": (_i, [C.POINTER(StepArgs)]),
    "qd_graph_create": (_i, [C.POINTER(StepArgs), _i, _vp, C.POINTER(_vp)]),
    "qd_graph_launch": (_i, [_vp, _vp]),
    "qd_graph_destroy": (_i, [_vp]),
    "qd_check_device_error": (_i, [_vp, C.POINTER(_i)]),
    "qd_verify_workspace_bytes": (_sz, [C.POINTER(StepArgs), _i]),
    "qd_verify_step": (_i, [C.POINTER(StepArgs), _vp, _i, _vp, _vp, _vp, _vp]),
    "qd_prefill_workspace_bytes": (_sz, [C.POINTER(StepArgs), _i]),
    "qd_prefill": (_i, [C.POINTER(StepArgs), _vp, _i, _vp, _vp]),
    "qd_debug_wait_timeout": (_i, [_i, _vp]),
    "qd_gemv_w4_workspace_bytes": (_sz, [_i, _i]),
    "qd_gemv_w4_ex": (_i, [_vp, _vp, _i, _i, _vp, _vp, _vp, _sz, _vp]),
    "qd_debug_q8_block_dots": (_i, [_vp, _vp, _i, _i, _vp, _vp, _vp, _vp, _vp]),
    "qd_debug_paged_indices": (_i, [_vp, _i, _i, _i, _i, _i, _vp, _vp]),
}

_lib = None


def lib():
    """Load libqd.so once; raise if it is missing (no CPU fallback exists)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run transformer_decode_step_weight_gb300.build")
        L = C.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of the functions include/qd.h declares."""
    src = open(HEADER).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(qd_[a-z0-9_]+)\s*\(", src)))


class QDError(RuntimeError):
    pass


def _check(rc: int):
    if rc != QD_OK:
        raise QDError(f"libqd error {rc}: {lib().qd_last_error().decode()}")


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _p(t):
    return None if t is None else t.data_ptr()


# ---------------------------------------------------------------- single ops


def gemv_bf16(W, x, y=None, stream=None):
    """y[b] = W @ x[b]; W bf16 [R, K]; x bf16 or f32 [B, K] -> f32 [B, R]."""
    x2 = x if x.dim() == 2 else x.reshape(1, -1)
    R, K = W.shape
    if y is None:
        y = torch.empty((x2.shape[0], R), dtype=torch.float32, device=W.device)
    _check(lib().qd_gemv_bf16(_p(W), R, K, _p(x2), int(x2.dtype == torch.float32), _p(y), x2.shape[0],
                              _stream(stream)))
    return y


def gemv_q8_0(qs, d, x=None, xq=None, xd=None, act=QD_ACT_F32, y=None, stream=None):
    R, K = qs.shape
    if y is None:
        y = torch.empty(R, dtype=torch.float32, device=qs.device)
    _check(lib().qd_gemv_q8_0(_p(qs), _p(d), R, K, _p(x), _p(xq), _p(xd), act, _p(y), _stream(stream)))
    return y


def debug_wait_timeout(limit_us: int, stream=None):
    """Run a bounded wait that nothing completes (QD_DEVERR_TIMEOUT afterwards)."""
    _check(lib().qd_debug_wait_timeout(int(limit_us), _stream(stream)))


def gemv_w4_workspace_bytes(R: int, K: int) -> int:
    return int(lib().qd_gemv_w4_workspace_bytes(R, K))


def gemv_w4(W, d, x, y=None, workspace=None, stream=None):
    """y = (d * q) @ x; W packed uint8 [R, K / 2], d f16 [R], x bf16 [K] -> f32 [R].
    `workspace` (zero-filled uint8, gemv_w4_workspace_bytes) lets small matrices split K."""
    R, Kh = W.shape
    if y is None:
        y = torch.empty(R, dtype=torch.float32, device=W.device)
    if workspace is None:
        _check(lib().qd_gemv_w4(_p(W), _p(d), R, 2 * Kh, _p(x), _p(y), _stream(stream)))
    else:
        _check(lib().qd_gemv_w4_ex(_p(W), _p(d), R, 2 * Kh, _p(x), _p(y), _p(workspace), workspace.numel(),
                                   _stream(stream)))
    return y


def gemv_w4_topk(W, d, x, k, y=None, workspace=None, stream=None):
    """(logits, top-k ids, top-k values) of the INT4 LM-head form."""
    R, Kh = W.shape
    if y is None:
        y = torch.empty(R, dtype=torch.float32, device=W.device)
    if workspace is None:
        workspace = torch.zeros(int(lib().qd_w4_topk_workspace_bytes()), dtype=torch.uint8, device=W.device)
    ids = torch.empty(k, dtype=torch.int32, device=W.device)
    vals = torch.empty(k, dtype=torch.float32, device=W.device)
    _check(lib().qd_gemv_w4_topk(_p(W), _p(d), R, 2 * Kh, _p(x), k, _p(y), _p(ids), _p(vals), _p(workspace),
                                 workspace.numel(), _stream(stream)))
    return y, ids, vals


def gemm_workspace_bytes(rows, cols, wtype=QD_W_Q8_0):
    return int(lib().qd_gemm_workspace_bytes(rows, cols, wtype))


def gemm_q8_0(qs, d, x, y=None, workspace=None, stream=None):
    """y[b] = bf16(f32(d) * qs) @ x[b] on the tensor cores; x bf16 [B, K] -> f32 [B, R]."""
    R, K = qs.shape
    B = x.shape[0]
    if y is None:
        y = torch.empty((B, R), dtype=torch.float32, device=qs.device)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().qd_gemm_q8_0(_p(qs), _p(d), R, K, _p(x), B, _p(y), _p(workspace), nbytes, _stream(stream)))
    return y


def quantize_q8_0(x, stream=None):
    n = x.numel()
    xq = torch.empty(n, dtype=torch.int8, device=x.device)
    xd = torch.empty(n // 32, dtype=torch.float16, device=x.device)
    _check(lib().qd_quantize_q8_0(_p(x), n, _p(xq), _p(xd), _stream(stream)))
    return xq, xd


def attn_workspace_bytes(batch, hq, hkv, max_ctx):
    return int(lib().qd_attn_workspace_bytes(batch, hq, hkv, max_ctx))


def attn_decode_paged(q, k_pages, v_pages, page_table, seq_lens, scale, out=None, workspace=None, stream=None):
    """q f32 [B, Hq, D]; caches bf16 [n_pages, Hkv, ps, D]; page_table int32 [B, max_pages]."""
    B, Hq, D = q.shape
    n_pages, Hkv, ps, _ = k_pages.shape
    max_pages = page_table.shape[1]
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = torch.zeros(attn_workspace_bytes(B, Hq, Hkv, max_pages * ps), dtype=torch.uint8,
                                device=q.device)
    _check(lib().qd_attn_decode_paged(_p(q), _p(k_pages), _p(v_pages), _p(page_table), _p(seq_lens), B, Hq, Hkv,
                                      D, ps, max_pages, n_pages, float(scale), _p(out), _p(workspace),
                                      workspace.numel(), _stream(stream)))
    return out


def attn_decode_paged_noalloc(q, k_pages, v_pages, page_table, seq_lens, scale, out=None, stream=None):
    """qd_attn_decode_paged with the library's static scratch instead of a workspace."""
    B, Hq, D = q.shape
    n_pages, Hkv, ps, _ = k_pages.shape
    if out is None:
        out = torch.empty_like(q)
    _check(lib().qd_attn_decode_paged_noalloc(_p(q), _p(k_pages), _p(v_pages), _p(page_table), _p(seq_lens), B,
                                              Hq, Hkv, D, ps, page_table.shape[1], n_pages, float(scale), _p(out),
                                              _stream(stream)))
    return out


# The serving calls below run many times per token, so their checks stay cheap: no context is
# entered where the tensors' device is current and no stream is given.
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _raw_stream(device: int):
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return get(device) if get is not None else torch.cuda.current_stream(device).cuda_stream


def _elsewhere(t, stream):
    """None where t's device is current and no stream is given; else a context that makes both
    current, so that what a call allocates belongs to the stream that its kernels run on."""
    dev = t.get_device()
    if stream is None:
        return None if dev < 0 or _current_device() == dev else torch.cuda.device(dev)
    if dev >= 0 and stream.device.index != dev:
        raise ValueError(f"stream on {stream.device}, tensors on cuda:{dev}")
    return torch.cuda.stream(stream)


def _want(name, t, dtype, dims, device, shape=None):
    """Refuses a tensor that the C entry could not take as it is (contiguous, on CUDA device `device`)."""
    if (t.dtype is dtype and t.get_device() == device >= 0 and t.dim() == dims and t.is_contiguous()
            and (shape is None or t.shape == shape)):
        return
    if device < 0 or t.get_device() != device:
        raise ValueError(f"{name}: on {t.device}, expected the first tensor's device, a CUDA device")
    if t.dtype != dtype or t.dim() != dims or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dims}-dimensional {dtype} tensor, got {t.dtype} {tuple(t.shape)}")
    raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _rows(fn, q, k_pages, v_pages, page_table, seq_lens, cu, out):
    """The common checks of attn_prompt and attn_decode_shared."""
    dev = q.get_device()
    if q.dim() != 3 or q.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"{fn}: q must be [rows, heads, head_dim] in float32 or bfloat16")
    n, hq, d = q.shape
    s0, s1, s2 = q.stride()
    if n and (s2 != 1 or (s1 != d and hq > 1)):
        raise ValueError(f"{fn}: a row's heads must be contiguous (strides {q.stride()})")
    _want("k_pages", k_pages, torch.bfloat16, 4, dev)
    _want("v_pages", v_pages, torch.bfloat16, 4, dev, k_pages.shape)
    if k_pages.shape[3] != d:
        raise ValueError(f"{fn}: head_dim {d} and {k_pages.shape[3]}")
    _want("page_table", page_table, torch.int32, 2, dev)
    _want("seq_lens", seq_lens, torch.int32, 1, dev, page_table.shape[:1])
    _want("segment starts", cu, torch.int32, 1, dev)
    if out is not None:
        _want("out", out, q.dtype, 3, dev, q.shape)
    return s0 if n > 1 else hq * d


# What of a workspace has to be zero before its first use (QD_ATTN_WORKSPACE_HEAD in qd.h)
_ATTN_HEAD = 8192


def _scratch(workspace, nbytes, t, head):
    if workspace is None:
        workspace = torch.empty(nbytes(), dtype=torch.uint8, device=t.device)
        workspace[:head].zero_()
        return workspace
    _want("workspace", workspace, torch.uint8, 1, t.get_device())
    return workspace


def attn_prompt_workspace_bytes() -> int:
    return int(lib().qd_attn_prompt_workspace_bytes())


def attn_prompt(q, k_pages, v_pages, page_table, cu_rows, seq_lens, scale, out=None, workspace=None, stream=None):
    """Causal attention over the packed rows of several prompts: q f32 or bf16 [rows, Hq, D] (rows may be
    strided), sequence b's rows cu_rows[b] .. cu_rows[b + 1), the last of them at position seq_lens[b] - 1;
    caches bf16 [n_pages, Hkv, ps, D] with the rows' K/V written. -> [rows, Hq, D] of q's type."""
    away = _elsewhere(q, stream)
    if away is not None:
        with away:
            return attn_prompt(q, k_pages, v_pages, page_table, cu_rows, seq_lens, scale, out, workspace)
    q_stride = _rows("attn_prompt", q, k_pages, v_pages, page_table, seq_lens, cu_rows, out)
    n, Hq, D = q.shape
    B, max_pages = page_table.shape
    n_pages, Hkv, ps, _ = k_pages.shape
    if cu_rows.shape[0] != B + 1:
        raise ValueError(f"attn_prompt: {cu_rows.numel()} segment starts for {B} sequences")
    if out is None:
        out = torch.empty((n, Hq, D), dtype=q.dtype, device=q.device)
    if n == 0:
        return out
    workspace = _scratch(workspace, attn_prompt_workspace_bytes, q, _ATTN_HEAD)
    _check(lib().qd_attn_prompt(q.data_ptr(), q.dtype is torch.float32, q_stride, k_pages.data_ptr(),
                                v_pages.data_ptr(), page_table.data_ptr(), cu_rows.data_ptr(), seq_lens.data_ptr(),
                                B, n, Hq, Hkv, D, ps, max_pages, n_pages, scale, out.data_ptr(),
                                workspace.data_ptr(), workspace.numel(), _raw_stream(q.get_device())))
    return out


def attn_shared_workspace_bytes(batch: int, hq: int, hkv: int) -> int:
    return int(lib().qd_attn_shared_workspace_bytes(batch, hq, hkv))


def attn_decode_shared(q, k_pages, v_pages, page_table, seq_lens, cu_seqs, shared_lens, scale, out=None,
                       workspace=None, stream=None):
    """attn_decode_paged for sequences that share prefixes: group i is the sequences cu_seqs[i] ..
    cu_seqs[i + 1), whose first shared_lens[i] tokens lie in the same pages (read once per group).
    q f32 or bf16 [B, Hq, D] -> [B, Hq, D] of q's type."""
    away = _elsewhere(q, stream)
    if away is not None:
        with away:
            return attn_decode_shared(q, k_pages, v_pages, page_table, seq_lens, cu_seqs, shared_lens, scale, out,
                                      workspace)
    q_stride = _rows("attn_decode_shared", q, k_pages, v_pages, page_table, seq_lens, cu_seqs, out)
    B, Hq, D = q.shape
    n_pages, Hkv, ps, _ = k_pages.shape
    _want("shared_lens", shared_lens, torch.int32, 1, q.get_device())
    groups = shared_lens.shape[0]
    if page_table.shape[0] != B or cu_seqs.shape[0] != groups + 1:
        raise ValueError(f"attn_decode_shared: {page_table.shape[0]} page tables for {B} rows, {cu_seqs.numel()} "
                         f"group starts for {groups} lengths")
    if out is None:
        out = torch.empty((B, Hq, D), dtype=q.dtype, device=q.device)
    if B == 0:
        return out
    workspace = _scratch(workspace, lambda: attn_shared_workspace_bytes(B, Hq, Hkv), q, _ATTN_HEAD)
    _check(lib().qd_attn_decode_shared(q.data_ptr(), q.dtype is torch.float32, q_stride, k_pages.data_ptr(),
                                       v_pages.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(),
                                       cu_seqs.data_ptr(), shared_lens.data_ptr(), groups, B, Hq, Hkv, D, ps,
                                       page_table.shape[1], n_pages, scale, out.data_ptr(), workspace.data_ptr(),
                                       workspace.numel(), _raw_stream(q.get_device())))
    return out


def verify_sample_workspace_bytes(batch: int) -> int:
    return int(lib().qd_verify_sample_workspace_bytes(batch))


def verify_sample(target_probs, draft_probs, draft, u, tok, pos, step, out_tokens, n_draft=None, n_accept=None,
                  workspace=None, stream=None):
    """Sampled verification of drafts: target_probs f32 [B, k, V], draft_probs f32 [B, k - 1, V] (rows may be
    padded), draft int32 [B, k - 1], u f32 [B, k]. Advances tok, pos, step [B] and out_tokens [B, max_steps] and
    returns n_accept int32 [B]."""
    fn = "verify_sample"
    away = _elsewhere(target_probs, stream)
    if away is not None:
        with away:
            return verify_sample(target_probs, draft_probs, draft, u, tok, pos, step, out_tokens, n_draft, n_accept,
                                 workspace)
    if target_probs.dim() != 3 or target_probs.dtype != torch.float32:
        raise ValueError(f"{fn}: target_probs must be float32 [B, k, V]")
    B, k, V = target_probs.shape
    dev = target_probs.get_device()
    t_stride = _row_stride("target_probs", target_probs, B, k, V, dev)
    d_stride = _row_stride("draft_probs", draft_probs, B, k - 1, V, dev) if k > 1 else V
    if k > 1:
        _want("draft", draft, torch.int32, 2, dev, (B, k - 1))
    _want("u", u, torch.float32, 2, dev, (B, k))
    one = (B,)
    _want("tok", tok, torch.int32, 1, dev, one)
    _want("pos", pos, torch.int32, 1, dev, one)
    _want("step", step, torch.int32, 1, dev, one)
    if n_draft is not None:
        _want("n_draft", n_draft, torch.int32, 1, dev, one)
    if n_accept is not None:
        _want("n_accept", n_accept, torch.int32, 1, dev, one)
    else:
        n_accept = torch.empty(B, dtype=torch.int32, device=target_probs.device)
    _want("out_tokens", out_tokens, torch.int32, 2, dev)
    if out_tokens.shape[0] != B:
        raise ValueError(f"{fn}: out_tokens has {out_tokens.shape[0]} rows for {B} sequences")
    if B == 0:
        return n_accept
    workspace = _scratch(workspace, lambda: verify_sample_workspace_bytes(B), target_probs, 4 * B)
    _check(lib().qd_verify_sample(target_probs.data_ptr(), t_stride, draft_probs.data_ptr() if k > 1 else None,
                                  d_stride, draft.data_ptr() if k > 1 else None, _p(n_draft), u.data_ptr(), V, B, k,
                                  tok.data_ptr(), pos.data_ptr(), step.data_ptr(), out_tokens.data_ptr(),
                                  out_tokens.shape[1], n_accept.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                  _raw_stream(dev)))
    return n_accept


def _row_stride(name, t, B, rows, V, dev):
    """Elements from one row of f32 [B, rows, V] to the next; the rows must be evenly spaced."""
    if t.dtype is not torch.float32 or t.get_device() != dev or t.shape != (B, rows, V):
        raise ValueError(f"verify_sample: {name} must be float32 {(B, rows, V)} on the first tensor's device")
    s0, s1, s2 = t.stride()
    s = s1 if rows > 1 else (s0 if B > 1 else V)
    if t.numel() and (s2 != 1 and V > 1 or (B > 1 and s0 != rows * s)):
        raise ValueError(f"verify_sample: {name}'s rows must be evenly spaced (strides {t.stride()})")
    return s


# A window that hides nothing, and what of the workspaces of the windowed decode and of key weights has
# to be zero before their first use (QD_ATTN_WINDOW_HEAD, QD_ATTN_WEIGHTS_HEAD in qd.h)
ALL_KEYS = 2 ** 31 - 1
_WINDOW_HEAD = 16384


def _counts(fn, **values):
    """Refuses numbers that a 32-bit argument would not hold as they are (the others the library refuses)."""
    for name, n in values.items():
        if not -ALL_KEYS <= n <= ALL_KEYS:
            raise ValueError(f"{fn}: {name}={n}")


def attn_prompt_window(q, k_pages, v_pages, page_table, cu_rows, seq_lens, scale, window=None, n_sinks=0, out=None,
                       workspace=None, stream=None):
    """attn_prompt in which each row sees its last `window` tokens (itself among them; None: all) and the first
    n_sinks; the other arguments and the workspace are attn_prompt's."""
    away = _elsewhere(q, stream)
    if away is not None:
        with away:
            return attn_prompt_window(q, k_pages, v_pages, page_table, cu_rows, seq_lens, scale, window, n_sinks, out,
                                      workspace)
    fn = "attn_prompt_window"
    q_stride = _rows(fn, q, k_pages, v_pages, page_table, seq_lens, cu_rows, out)
    n, Hq, D = q.shape
    B, max_pages = page_table.shape
    n_pages, Hkv, ps, _ = k_pages.shape
    if cu_rows.shape[0] != B + 1:
        raise ValueError(f"{fn}: {cu_rows.numel()} segment starts for {B} sequences")
    window = ALL_KEYS if window is None else window
    if not (0 < window <= ALL_KEYS and 0 <= n_sinks <= ALL_KEYS):
        _counts(fn, window=window, n_sinks=n_sinks)
    if out is None:
        out = torch.empty((n, Hq, D), dtype=q.dtype, device=q.device)
    if n == 0:
        return out
    workspace = _scratch(workspace, attn_prompt_workspace_bytes, q, _ATTN_HEAD)
    _check(lib().qd_attn_prompt_window(q.data_ptr(), q.dtype is torch.float32, q_stride, k_pages.data_ptr(),
                                       v_pages.data_ptr(), page_table.data_ptr(), cu_rows.data_ptr(),
                                       seq_lens.data_ptr(), B, n, Hq, Hkv, D, ps, max_pages, n_pages, scale,
                                       window, n_sinks, out.data_ptr(),
                                       workspace.data_ptr(), workspace.numel(), _raw_stream(q.get_device())))
    return out


def attn_decode_window_workspace_bytes(batch: int, hq: int, hkv: int, max_keys: int = 0) -> int:
    """max_keys: min(window + n_sinks, a page-table row's tokens) where key_weights are asked for, else 0."""
    return int(lib().qd_attn_decode_window_workspace_bytes(batch, hq, hkv, max_keys))


def attn_decode_window(q, k_pages, v_pages, page_table, seq_lens, scale, window=None, n_sinks=0, key_weights=None,
                       out=None, workspace=None, stream=None):
    """Decode attention in which each row sees its last `window` tokens (None: all) and the first n_sinks: q f32 or
    bf16 [B, Hq, D] -> [B, Hq, D] of q's type. key_weights f32 [B, Hkv, max_pages * ps]: each visible key's softmax
    weight, summed over its kv head's q heads, is added to it."""
    fn = "attn_decode_window"
    away = _elsewhere(q, stream)
    if away is not None:
        with away:
            return attn_decode_window(q, k_pages, v_pages, page_table, seq_lens, scale, window, n_sinks, key_weights, out,
                                      workspace)
    dev = q.get_device()
    q_stride = _rows(fn, q, k_pages, v_pages, page_table, seq_lens, seq_lens, out)
    B, Hq, D = q.shape
    n_pages, Hkv, ps, _ = k_pages.shape
    max_pages = page_table.shape[1]
    if page_table.shape[0] != B:
        raise ValueError(f"{fn}: {page_table.shape[0]} page tables for {B} rows")
    window = ALL_KEYS if window is None else window
    if not (0 < window <= ALL_KEYS and 0 <= n_sinks <= ALL_KEYS):
        _counts(fn, window=window, n_sinks=n_sinks)
    keys = 0
    if key_weights is not None:
        _want("key_weights", key_weights, torch.float32, 3, dev, (B, Hkv, max_pages * ps))
        keys = min(window + n_sinks, max_pages * ps)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=q.dtype, device=q.device)
    if B == 0:
        return out
    workspace = _scratch(workspace, lambda: attn_decode_window_workspace_bytes(B, Hq, Hkv, keys), q, _WINDOW_HEAD)
    _check(lib().qd_attn_decode_window(q.data_ptr(), q.dtype is torch.float32, q_stride, k_pages.data_ptr(),
                                       v_pages.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(), B, Hq, Hkv, D,
                                       ps, max_pages, n_pages, scale, window, n_sinks, _p(key_weights), out.data_ptr(),
                                       workspace.data_ptr(), workspace.numel(), _raw_stream(dev)))
    return out


def attn_key_weights_workspace_bytes(batch: int, rows: int, hq: int, hkv: int, last: int = 0,
                                     dtype=torch.float32) -> int:
    """dtype: q's type (float32's size, three times bfloat16's, serves either)."""
    if dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"attn_key_weights: dtype {dtype}, expected float32 or bfloat16")
    return int(lib().qd_attn_key_weights_workspace_bytes_for(dtype is torch.float32, batch, rows, hq, hkv, last))


def attn_key_weights(q, k_pages, page_table, cu_rows, seq_lens, scale, key_weights, last=0, window=None, n_sinks=0,
                     workspace=None, stream=None):
    """Adds to key_weights f32 [B, Hkv, max_pages * ps] the softmax weights that attn_prompt (attn_prompt_window) of
    these rows gives to each key, summed over the last `last` rows of each sequence (0: all) and the q heads of a kv
    head. Returns key_weights."""
    fn = "attn_key_weights"
    away = _elsewhere(q, stream)
    if away is not None:
        with away:
            return attn_key_weights(q, k_pages, page_table, cu_rows, seq_lens, scale, key_weights, last, window, n_sinks,
                                    workspace)
    dev = q.get_device()
    q_stride = _rows(fn, q, k_pages, k_pages, page_table, seq_lens, cu_rows, None)
    n, Hq, D = q.shape
    B, max_pages = page_table.shape
    n_pages, Hkv, ps, _ = k_pages.shape
    if cu_rows.shape[0] != B + 1:
        raise ValueError(f"{fn}: {cu_rows.numel()} segment starts for {B} sequences")
    _want("key_weights", key_weights, torch.float32, 3, dev, (B, Hkv, max_pages * ps))
    window = ALL_KEYS if window is None else window
    if not (0 < window <= ALL_KEYS and 0 <= n_sinks <= ALL_KEYS and 0 <= last <= ALL_KEYS):
        _counts(fn, window=window, n_sinks=n_sinks, last=last)
    if n == 0:
        return key_weights
    workspace = _scratch(workspace, lambda: attn_key_weights_workspace_bytes(B, n, Hq, Hkv, last, q.dtype), q,
                         _WINDOW_HEAD)
    _check(lib().qd_attn_key_weights(q.data_ptr(), q.dtype is torch.float32, q_stride, k_pages.data_ptr(),
                                     page_table.data_ptr(), cu_rows.data_ptr(), seq_lens.data_ptr(), B, n, Hq, Hkv, D,
                                     ps, max_pages, n_pages, scale, last, window, n_sinks,
                                     key_weights.data_ptr(), workspace.data_ptr(), workspace.numel(), _raw_stream(dev)))
    return key_weights


def qk_norm_rope(qkv, q_norm, k_norm, rope, k_pages, v_pages, page_table, cu_rows, seq_lens, eps, positions=None,
                 axes=None, cast=False, out=None, dtype=None, stream=None):
    """The q and k heads of packed rows normed and rotated, K and V written to their cache slots: qkv f32 or bf16
    [rows, (Hq + 2 Hkv) * 128] (rows may be strided), sequence b's rows cu_rows[b] .. cu_rows[b + 1), the last of
    them at slot seq_lens[b] - 1. rope: rope_table(...). positions int32 [axes, rows] (None: the slots), axes: the
    position axis of each of the 64 frequencies. cast: bf16 after the division and the weight, as a BF16 model's
    decode step. -> q [rows, Hq, 128] of `dtype` (default: qkv's)."""
    fn = "qk_norm_rope"
    away = _elsewhere(qkv, stream)
    if away is not None:
        with away:
            return qk_norm_rope(qkv, q_norm, k_norm, rope, k_pages, v_pages, page_table, cu_rows, seq_lens, eps,
                                positions, axes, cast, out, dtype)
    dev = qkv.get_device()
    if qkv.dim() != 2 or qkv.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"{fn}: qkv must be [rows, heads * 128] in float32 or bfloat16")
    n, width = qkv.shape
    if n and qkv.stride(1) != 1:
        raise ValueError(f"{fn}: a row's heads must be contiguous (strides {qkv.stride()})")
    _want("k_pages", k_pages, torch.bfloat16, 4, dev)
    _want("v_pages", v_pages, torch.bfloat16, 4, dev, k_pages.shape)
    n_pages, Hkv, ps, D = k_pages.shape
    Hq = width // D - 2 * Hkv if D else 0
    if Hq < 1 or width % D:
        raise ValueError(f"{fn}: rows of {width} for {Hkv} kv heads of {D}")
    _want("q_norm", q_norm, torch.bfloat16, 1, dev, (D,))
    _want("k_norm", k_norm, torch.bfloat16, 1, dev, (D,))
    _want("rope", rope, torch.float32, 3, dev)
    rope_max, half, two = rope.shape
    if 2 * half != D or two != 2:
        raise ValueError(f"{fn}: rope table {tuple(rope.shape)}, expected [positions, {D // 2}, 2]")
    _want("page_table", page_table, torch.int32, 2, dev)
    B, max_pages = page_table.shape
    _want("seq_lens", seq_lens, torch.int32, 1, dev, (B,))
    _want("segment starts", cu_rows, torch.int32, 1, dev, (B + 1,))
    n_axes = 1
    if positions is not None:
        if positions.dim() == 1:
            positions = positions[None]
        _want("positions", positions, torch.int32, 2, dev)
        n_axes = positions.shape[0]
        if positions.shape[1] != n:
            raise ValueError(f"{fn}: {positions.shape[1]} positions for {n} rows")
    if axes is not None:
        axes = bytes(axes)
        if len(axes) != D // 2:
            raise ValueError(f"{fn}: axes of {len(axes)} frequencies, expected {D // 2}")
    if out is None:
        out = torch.empty((n, Hq, D), dtype=dtype or qkv.dtype, device=qkv.device)
    elif out.dtype not in (torch.float32, torch.bfloat16) or (dtype is not None and dtype != out.dtype):
        raise ValueError(f"{fn}: out in {out.dtype}, expected {dtype or 'float32 or bfloat16'}")
    _want("out", out, out.dtype, 3, dev, (n, Hq, D))
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"{fn}: dtype {out.dtype}, expected float32 or bfloat16")
    if n == 0:
        return out
    _check(lib().qd_qk_norm_rope(qkv.data_ptr(), qkv.dtype is torch.float32, qkv.stride(0) if n > 1 else width,
                                 q_norm.data_ptr(), k_norm.data_ptr(), eps, bool(cast), rope.data_ptr(), rope_max,
                                 _p(positions), n_axes, axes, page_table.data_ptr(), cu_rows.data_ptr(),
                                 seq_lens.data_ptr(), B, n, Hq, Hkv, D, ps, max_pages, n_pages, out.data_ptr(),
                                 out.dtype is torch.float32, k_pages.data_ptr(), v_pages.data_ptr(), _raw_stream(dev)))
    return out


class PageCache:
    """Page operations on the K/V caches of all layers (bf16 [n_pages, Hkv, ps, D] each).

    ``page_table`` int32 [max_seqs, max_pages] (-1 past a sequence's pages), ``seq_lens`` int32
    [max_seqs] and ``refs`` int32 [n_pages] (how many entries name each page, 0: free) are the
    state, device tensors that the calls update; without them only ``copy`` works. ``empty``
    makes the state of an empty cache. One PageCache serves one stream at a time, and stays
    alive until the work of its calls is done (it owns their workspace).
    """

    def __init__(self, k_cache, v_cache, page_table=None, seq_lens=None, refs=None):
        if not k_cache or len(k_cache) != len(v_cache):
            raise ValueError(f"PageCache: {len(k_cache)} K and {len(v_cache)} V caches")
        self.k_cache, self.v_cache = list(k_cache), list(v_cache)
        first = self.k_cache[0]
        for t in self.k_cache + self.v_cache:
            _want("PageCache: a cache", t, torch.bfloat16, 4, first.get_device(), first.shape)
        self.device, self._dev = first.device, first.get_device()
        L = len(self.k_cache)
        a = PageCacheArgs()
        self._k_arr = (_vp * L)(*[_p(t) for t in self.k_cache])
        self._v_arr = (_vp * L)(*[_p(t) for t in self.v_cache])
        a.k_cache, a.v_cache = C.cast(self._k_arr, _vp), C.cast(self._v_arr, _vp)
        a.n_layers = L
        a.n_pages, a.n_kv_heads, a.page_size, a.head_dim = first.shape
        self.page_table, self.seq_lens, self.refs = page_table, seq_lens, refs
        if page_table is not None:
            _want("PageCache: page_table", page_table, torch.int32, 2, self._dev)
            _want("PageCache: seq_lens", seq_lens, torch.int32, 1, self._dev, page_table.shape[:1])
            _want("PageCache: refs", refs, torch.int32, 1, self._dev, first.shape[:1])
            a.page_table, a.seq_lens, a.refs = _p(page_table), _p(seq_lens), _p(refs)
            a.max_seqs, a.max_pages = page_table.shape
            self.workspace = torch.zeros(int(lib().qd_pages_workspace_bytes(C.byref(a))), dtype=torch.uint8,
                                         device=self.device)
            a.workspace, a.workspace_bytes = _p(self.workspace), self.workspace.numel()
        self.args = a
        self._ref = C.byref(a)

    @classmethod
    def empty(cls, k_cache, v_cache, max_seqs: int, max_pages: int):
        dev = k_cache[0].device
        return cls(k_cache, v_cache, torch.full((max_seqs, max_pages), -1, dtype=torch.int32, device=dev),
                   torch.zeros(max_seqs, dtype=torch.int32, device=dev),
                   torch.zeros(k_cache[0].shape[0], dtype=torch.int32, device=dev))

    def _list(self, name, t, n=None):
        _want(name, t, torch.int32, 1, self._dev, None if n is None else (n,))
        return t.data_ptr()

    def _run(self, stream, fn, *args):
        away = _elsewhere(self.k_cache[0], stream)
        if away is None:
            _check(fn(self._ref, *args, _raw_stream(self._dev)))
        else:
            with away:
                _check(fn(self._ref, *args, _raw_stream(self._dev)))

    def copy(self, src, dst, stream=None):
        """Page src[i] to page dst[i] in every layer's K and V (device int32 lists)."""
        n = src.numel()
        self._run(stream, lib().qd_pages_copy, self._list("src", src), self._list("dst", dst, n), n)

    def fork(self, parents, children, stream=None):
        """Sequence children[i] (empty) becomes a copy of parents[i], its pages shared."""
        n = parents.numel()
        self._run(stream, lib().qd_pages_fork, self._list("parents", parents), self._list("children", children, n), n)

    def extend(self, n_new, stream=None):
        """Pages for n_new[s] more tokens of each sequence; shared partial pages are copied."""
        self._run(stream, lib().qd_pages_extend, self._list("n_new", n_new, self.args.max_seqs))

    def trim(self, new_lens, stream=None):
        """Sequence s cut to new_lens[s] tokens (negative: unchanged; 0 frees it)."""
        self._run(stream, lib().qd_pages_trim, self._list("new_lens", new_lens, self.args.max_seqs))

    def compact(self, n_live=None, stream=None):
        """The pages in use moved to the lowest ids; returns their number (device int32 [1])."""
        if n_live is None:
            away = _elsewhere(self.k_cache[0], stream)
            if away is not None:
                with away:
                    return self.compact()
            n_live = torch.empty(1, dtype=torch.int32, device=self.device)
        self._run(stream, lib().qd_pages_compact, self._list("n_live", n_live, 1))
        return n_live

    def evict(self, key_weights, keep, n_sinks=0, n_recent=0, stream=None):
        """Sequence s cut to keep[s] tokens (negative or not below its length: unchanged): the first n_sinks, the last
        n_recent and those of the largest key_weights f32 [layers, max_seqs, Hkv, max_pages * ps], each layer and kv
        head its own. K, V and weights move down; weights past the kept ones become 0."""
        a = self.args
        _want("key_weights", key_weights, torch.float32, 4, self._dev,
              (a.n_layers, a.max_seqs, a.n_kv_heads, a.max_pages * a.page_size))
        if not (0 <= n_sinks <= ALL_KEYS and 0 <= n_recent <= ALL_KEYS):
            _counts("evict", n_sinks=n_sinks, n_recent=n_recent)
        self._run(stream, lib().qd_pages_evict, key_weights.data_ptr(), self._list("keep", keep, a.max_seqs), n_sinks,
                  n_recent)


def argmax_advance(logits, tok, pos, step, out_tokens, workspace=None, stream=None):
    B, V = logits.shape
    if workspace is None:
        workspace = torch.zeros(int(lib().qd_argmax_workspace_bytes(B)), dtype=torch.uint8, device=logits.device)
    _check(lib().qd_argmax_advance(_p(logits), V, B, _p(tok), _p(pos), _p(step), _p(out_tokens),
                                   out_tokens.shape[1], _p(workspace), workspace.numel(), _stream(stream)))


def rope_table(max_pos, head_dim, theta, device, stream=None):
    t = torch.empty((max_pos, head_dim // 2, 2), dtype=torch.float32, device=device)
    _check(lib().qd_rope_table_init(_p(t), max_pos, head_dim, float(theta), _stream(stream)))
    return t


def check_device_error(stream=None) -> int:
    bits = _i(0)
    _check(lib().qd_check_device_error(_stream(stream), C.byref(bits)))
    return bits.value


def debug_q8_block_dots(qs, d, xq, xd, stream=None):
    """(int32 block dots [R, K/32], f32 y [R]) of the production i8-lane Q8_0 GEMV."""
    R, K = qs.shape
    dots = torch.empty((R, K // 32), dtype=torch.int32, device=qs.device)
    y = torch.empty(R, dtype=torch.float32, device=qs.device)
    _check(lib().qd_debug_q8_block_dots(_p(qs), _p(d), R, K, _p(xq), _p(xd), _p(dots), _p(y), _stream(stream)))
    return dots, y


def debug_paged_indices(page_table, page_size, n_tokens, n_pages=None, stream=None):
    B, max_pages = page_table.shape
    if n_pages is None:
        n_pages = max_pages * B
    idx = torch.empty((B, n_tokens), dtype=torch.int32, device=page_table.device)
    _check(lib().qd_debug_paged_indices(_p(page_table), B, max_pages, page_size, n_pages, n_tokens, _p(idx),
                                        _stream(stream)))
    return idx


# ---------------------------------------------------------------- whole step


class Decoder:
    """Owns the layer handles, step state and workspace of one decode run.

    ``model`` holds device tensors (see ``synth.ModelTensors``): per-layer
    weights, embedding, final norm, LM head, the per-layer K/V caches, page
    table, cached lengths and start tokens. The state buffers (tok, pos, step,
    out_tokens) are device int32 tensors advanced by the library.
    """

    def __init__(self, model, max_steps: int, act: int = QD_ACT_F32, lm_act: int | None = None,
                 device="cuda", verify_k: int = 0, top_k: int = 0, prefill_max: int = 0):
        self.m = model
        s = model.shape
        self.device = torch.device(device)
        wt = {"bf16": QD_W_BF16, "q8_0": QD_W_Q8_0, "int4": QD_W_INT4}[model.wtype]
        dims = LayerDims(s.hidden, s.n_q_heads, s.n_kv_heads, s.head_dim, s.ffn, s.rms_eps, s.rope_theta,
                         wt, act)
        self._handles = []
        for lt in model.layers:
            w = LayerWeights(_p(lt.w_qkv), _p(lt.w_o), _p(lt.w_gu), _p(lt.w_down),
                             _p(lt.s_qkv), _p(lt.s_o), _p(lt.s_gu), _p(lt.s_down),
                             _p(lt.ln_in), _p(lt.ln_post), _p(lt.q_norm), _p(lt.k_norm))
            h = _vp()
            _check(lib().qd_create_layer(C.byref(dims), C.byref(w), C.byref(h)))
            self._handles.append(h)
        L = len(self._handles)
        self._layer_arr = (_vp * L)(*[h.value for h in self._handles])
        self._k_arr = (_vp * L)(*[_p(t) for t in model.k_cache])
        self._v_arr = (_vp * L)(*[_p(t) for t in model.v_cache])
        B = int(model.start_tok.numel())
        self.batch = B
        self.max_steps = max_steps
        self.tok = model.start_tok.clone().to(torch.int32)
        self.pos = model.seq_lens.clone().to(torch.int32)
        self.step_ctr = torch.zeros(B, dtype=torch.int32, device=self.device)
        self.out_tokens = torch.full((B, max_steps), -1, dtype=torch.int32, device=self.device)
        self.logits = torch.empty((B, s.vocab), dtype=torch.float32, device=self.device)
        cap = model.max_pages * model.page_size
        self.rope = rope_table(cap, s.head_dim, s.rope_theta, self.device)
        n_pages = int(model.k_cache[0].shape[0])
        a = StepArgs()
        a.layers = C.cast(self._layer_arr, _vp)
        a.n_layers = L
        a.embed = _p(model.embed)
        a.final_norm = _p(model.final_norm)
        a.lm_head = _p(model.lm_head)
        a.lm_head_scales = _p(model.lm_head_scales)
        a.lm_act = act if lm_act is None else lm_act
        a.vocab = s.vocab
        a.k_cache = C.cast(self._k_arr, _vp)
        a.v_cache = C.cast(self._v_arr, _vp)
        a.page_table = _p(model.page_table)
        a.page_size = model.page_size
        a.max_pages = model.max_pages
        a.n_pages = n_pages
        a.rope_table = _p(self.rope)
        a.rope_max_pos = cap
        a.tok, a.pos, a.step, a.out_tokens = _p(self.tok), _p(self.pos), _p(self.step_ctr), _p(self.out_tokens)
        a.max_steps = max_steps
        a.batch = B
        a.logits = _p(self.logits)
        a.lm_wtype = QD_W_INT4 if model.lm_head.dtype == torch.uint8 else QD_W_BF16
        a.top_k = top_k
        if top_k:
            self.topk_ids = torch.full((top_k,), -1, dtype=torch.int32, device=self.device)
            self.topk_vals = torch.zeros(top_k, dtype=torch.float32, device=self.device)
            a.topk_ids, a.topk_vals = _p(self.topk_ids), _p(self.topk_vals)
        self.args = a
        nbytes = int(lib().qd_step_workspace_bytes(C.byref(a)))
        if verify_k:  # room for speculative verify passes of up to verify_k tokens
            nbytes = max(nbytes, int(lib().qd_verify_workspace_bytes(C.byref(a), verify_k)))
            self.verify_logits = torch.empty((verify_k, s.vocab), dtype=torch.float32, device=self.device)
            self.verify_target = torch.zeros(verify_k, dtype=torch.int32, device=self.device)
            self.n_accept = torch.zeros(1, dtype=torch.int32, device=self.device)
        if prefill_max:  # room for prompts of up to prefill_max tokens
            nbytes = max(nbytes, int(lib().qd_prefill_workspace_bytes(C.byref(a), prefill_max)))
            self.prefill_logits = torch.empty(s.vocab, dtype=torch.float32, device=self.device)
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
        a.workspace = _p(self.workspace)
        a.workspace_bytes = nbytes
        self._graph = None

    @property
    def launches_per_step(self) -> int:
        return int(lib().qd_step_launch_count(C.byref(self.args)))

    def residual(self) -> torch.Tensor:
        """The f32 residual stream [B, H] left in the workspace by the last step."""
        H = self.m.shape.hidden
        return self.workspace[: self.batch * H * 4].view(torch.float32).view(self.batch, H)

    def rows_residual(self, n: int) -> torch.Tensor:
        """The f32 residual rows [n, H] of the last verify pass or prefill (their scratch
        follows the decode step's workspace)."""
        H = self.m.shape.hidden
        off = int(lib().qd_step_workspace_bytes(C.byref(self.args)))
        return self.workspace[off: off + n * H * 4].view(torch.float32).view(n, H)

    def step(self, stream=None):
        _check(lib().qd_decode_step(C.byref(self.args), _stream(stream)))

    def verify(self, draft, stream=None):
        """One speculative verify pass over tok and the k - 1 draft tokens (device int32):
        fills verify_logits[:k], verify_target[:k] and n_accept, and advances the state."""
        k = int(draft.numel()) + 1
        _check(lib().qd_verify_step(C.byref(self.args), _p(draft) if k > 1 else None, k, _p(self.verify_logits),
                                    _p(self.verify_target), _p(self.n_accept), _stream(stream)))

    def prefill(self, tokens, stream=None):
        """The prompt `tokens` (device int32 [n]) at positions pos .. pos + n - 1 in one
        pass: writes their K/V, fills prefill_logits with the last row's logits and
        advances the state (tok = its argmax, pos += n, step += 1)."""
        _check(lib().qd_prefill(C.byref(self.args), _p(tokens), int(tokens.numel()), _p(self.prefill_logits),
                                _stream(stream)))

    def capture(self, steps_per_launch: int, stream=None):
        if self._graph is not None:
            lib().qd_graph_destroy(self._graph)
        g = _vp()
        _check(lib().qd_graph_create(C.byref(self.args), steps_per_launch, _stream(stream), C.byref(g)))
        self._graph = g
        self.graph_steps = steps_per_launch

    def replay(self, stream=None):
        _check(lib().qd_graph_launch(self._graph, _stream(stream)))

    def close(self):
        if self._graph is not None:
            lib().qd_graph_destroy(self._graph)
            self._graph = None
        for h in self._handles:
            lib().qd_destroy_layer(h)
        self._handles = []

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
