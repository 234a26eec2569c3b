"""Cases of the operators that fill and bound the K/V cache: norms and rotation of packed rows with their cache write,
attention with a sliding window and first tokens that stay visible (prompts, single tokens), the weights that attention
gives to each key, and eviction by them.

Shapes are those of the Qwen3-8B (32 q heads, 8 kv heads, 36 layers) and Qwen3-0.6B (16 q heads, 8 kv heads, 28 layers)
configurations of this repository; caches are bf16 [pages, kv heads, page size, 128]. The plain forms are elementary torch
operations in 32 bits; with `own` set, run() makes the framework's calls.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
D = 128
SCALE = 1.0 / math.sqrt(D)
EPS = 1e-6
THETA = 1e6
ALL = 2 ** 31 - 1      # a window that hides nothing


# ------------------------------------------------------------------------------------------------------ the cases


def listed():
    return [
        # one long document's projections, text and image tokens (three position axes), into the cache: the largest
        dict(name="rows-8192-3axes-bf16", op="rows", src="f32", dst="bf16", cast=True, axes=3, hq=32, hkv=8, page=64,
             batch=1, rows_lo=8192, rows_hi=8192, past_hi=0, lens=1),
        # one token of 64 conversations, all in 32 bits: latency
        dict(name="rows-64-tokens-f32", op="rows", src="f32", dst="f32", cast=False, axes=1, hq=32, hkv=8, page=16,
             batch=64, rows_lo=1, rows_hi=1, past_hi=4096, lens=2),
        # several users' messages behind their conversations, ragged
        dict(name="window-16-messages-bf16", op="prompt", dtype="bf16", hq=32, hkv=8, page=16, batch=16, rows_lo=20,
             rows_hi=700, past_hi=6000, window=1024, sinks=4, lens=3),
        # a long document from an empty cache: compute-bound
        dict(name="window-8192-bf16", op="prompt", dtype="bf16", hq=32, hkv=8, page=64, batch=1, rows_lo=8192,
             rows_hi=8192, past_hi=0, window=2048, sinks=64, lens=4),
        # the next chunk of three conversations, in the framework's own f32 rows; odd sizes
        dict(name="window-3-chunks-f32", op="prompt", dtype="f32", hq=16, hkv=8, page=16, batch=3, rows_lo=33,
             rows_hi=333, past_hi=12001, window=4099, sinks=5, lens=5),
        # the next token of 64 long conversations, f32 as the decode step's q
        dict(name="decode-64x4096-f32", op="decode", dtype="f32", hq=32, hkv=8, page=16, batch=64, len_hi=16384,
             window=4096, sinks=4, weights=False, lens=6),
        # one conversation's next token: latency
        dict(name="decode-1x1024-bf16", op="decode", dtype="bf16", hq=16, hkv=8, page=16, batch=1, len_hi=20000,
             window=1024, sinks=4, weights=False, lens=7),
        # the next token of 16 conversations, every key seen and its weight added up
        dict(name="decode-weights-16-f32", op="decode", dtype="f32", hq=32, hkv=8, page=16, batch=16, len_hi=8192,
             window=ALL, sinks=0, weights=True, lens=8),
        # the last 32 rows of eight prompts vote for the keys to keep
        dict(name="weights-8x32-bf16", op="weights", dtype="bf16", hq=32, hkv=8, page=16, batch=8, rows_lo=500,
             rows_hi=2000, past_hi=6000, last=32, window=ALL, sinks=0, lens=9),
        # every row of one prompt, in 32 bits
        dict(name="weights-2011-f32", op="weights", dtype="f32", hq=16, hkv=8, page=16, batch=1, rows_lo=2011,
             rows_hi=2011, past_hi=0, last=0, window=ALL, sinks=0, lens=10),
        # four long conversations cut to 1500 tokens each, in every layer
        dict(name="evict-4-of-36-layers", op="evict", layers=36, hkv=8, page=16, batch=4, len_hi=3300, keep=1500,
             sinks=4, recent=256, lens=11),
        # one conversation of the small model brought back under its budget: latency
        dict(name="evict-1-of-28-layers", op="evict", layers=28, hkv=8, page=16, batch=1, len_hi=1100, keep=1001,
             sinks=4, recent=64, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rows", "rows", "prompt", "prompt", "decode", "decode", "weights", "evict"])
    hq, hkv = rng.choice([(32, 8), (16, 8), (8, 8), (16, 2), (4, 2)])
    case = dict(op=op, hq=hq, hkv=hkv, page=rng.choice([16, 16, 32, 64, 128, 24, 7]), lens=rng.randrange(1 << 30))
    dtype = rng.choice(["bf16", "f32"])
    window, sinks = rng.choice([_log(rng, 1, 6000), ALL]), rng.choice([0, _log(rng, 1, 300)])
    if op == "evict":
        del case["hq"]
        n = _log(rng, 20, 3000)
        keep = rng.randint(max(1, n // 4), n)
        return dict(case, layers=rng.randint(1, 36), batch=_log(rng, 1, 4), len_hi=n, keep=keep,
                    sinks=rng.randint(0, keep // 4), recent=rng.randint(0, keep // 2))
    if op == "decode":
        batch = _log(rng, 1, 64)
        return dict(case, dtype=dtype, batch=batch, len_hi=_log(rng, 1, 200000 // batch), window=window, sinks=sinks,
                    weights=rng.random() < 0.5)
    batch = _log(rng, 1, 16)
    hi = _log(rng, 1, 4096 // batch + 40)
    case.update(batch=batch, rows_lo=rng.choice([0, 1, (hi + 1) // 2]), rows_hi=hi,
                past_hi=rng.choice([0, _log(rng, 1, 6000)]))
    if op == "rows":
        cast = rng.random() < 0.5
        return dict(case, src=rng.choice(["f32", "bf16"]), dst="bf16" if cast else dtype, cast=cast,
                    axes=rng.randint(1, 3))
    if op == "prompt":
        return dict(case, dtype=dtype, window=window, sinks=sinks)
    return dict(case, dtype=dtype, last=rng.choice([0, _log(rng, 1, 64)]), window=window, sinks=sinks)


def _lens(case):
    """The lengths of a case's sequences, from the case alone: (rows, tokens in the cache with them)."""
    r = random.Random(case["lens"])
    if "rows_hi" not in case:
        lens = [r.randint((case["len_hi"] + 1) // 2, case["len_hi"]) for _ in range(case["batch"])]
        return [1] * len(lens), lens
    rows = [r.randint(case["rows_lo"], case["rows_hi"]) for _ in range(case["batch"])]
    rows[-1] = max(rows[-1], 1)
    past = [r.randint(case["past_hi"] // 2, case["past_hi"]) for _ in rows]
    return rows, [n + p for n, p in zip(rows, past)]


# ------------------------------------------------------------------------------------------------------ the inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(generator=g)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _angles(positions):
    """(cos, sin) of each position and frequency, f32 [positions, D / 2, 2], from angles in 64 bits."""
    f = THETA ** (-2.0 * torch.arange(D // 2, dtype=torch.float64, device=DEV) / D)
    a = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).float()


def _axes(n):
    """The position axis that each of the 64 frequencies takes: sections as image and video tokens have them."""
    cuts = {1: [64], 2: [32, 32], 3: [16, 24, 24]}[n]
    return [a for a, m in enumerate(cuts) for _ in range(m)]


def prepare(case, seed):
    g, r, op = _gen(seed), random.Random(seed), case["op"]
    state = dict(case)
    page, hkv = case["page"], case["hkv"]
    rows, lens = _lens(case)
    need = [-(-n // page) for n in lens]
    width, pages = max(max(need), 1), sum(need) + 3
    perm = list(range(pages))
    r.shuffle(perm)
    ids = iter(perm)
    table = _ints([[next(ids) for _ in range(n)] + [-1] * (width - n) for n in need])
    state.update(n_rows=rows, cu=_ints(np.concatenate([[0], np.cumsum(rows)]).tolist()), max_rows=max(rows),
                 max_len=max(lens), cap=width * page, lens=_ints(lens), table=table)
    # values as a filled cache has them, N(0, 1)
    shape = (pages, hkv, page, D)
    if op == "evict":
        shape = (case["layers"],) + shape
        refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
        refs[table[table >= 0].long()] = 1
        # the table, lengths and counts in one tensor, so that a pass can start from the same ones
        state["first"] = torch.cat([table.flatten(), _ints(lens), refs])
        state["meta"] = state["first"].clone()
        B = case["batch"]
        state["table"] = state["meta"][:B * width].view(B, width)
        state["lens"] = state["meta"][B * width:B * width + B]
        state["refs"] = state["meta"][B * width + B:]
        state["keep"] = _ints([case["keep"]] * B)
        # few keys have most of the weight, some have none at all
        w = (2 * _normal(g, (case["layers"], B, hkv, width * page), torch.float32)).exp_()
        w.masked_fill_(torch.rand(w.shape, generator=g, device=DEV) < 0.1, 0.0)
        w.masked_fill_(torch.arange(width * page, device=DEV) >= state["lens"][:, None, None], 0.0)
        state["first_weights"], state["weights_now"] = w, w.clone()
    state["k"], state["v"] = _normal(g, shape, torch.bfloat16), _normal(g, shape, torch.bfloat16)
    if op == "evict":
        return state
    hq, total = case["hq"], sum(rows)
    if op == "rows":
        x = _normal(g, (total, (hq + 2 * hkv) * D), torch.float32) * 1.5
        # f32 rows are a projection's sums, bf16 ones have been rounded since
        state["x"] = x.bfloat16() if case["src"] == "bf16" else x
        state["q_norm"] = (1 + 0.1 * _normal(g, (D,), torch.float32)).bfloat16()
        state["k_norm"] = (1 + 0.1 * _normal(g, (D,), torch.float32)).bfloat16()
        state["angles"] = _angles(max(lens) + 64)
        state["axis_of"] = _axes(case["axes"])
        at = torch.cat([torch.arange(m - n, m, device=DEV) for n, m in zip(rows, lens)])
        # one axis: the tokens' slots. More: a token's row and column in its image beside its time
        state["positions"] = None if case["axes"] == 1 else torch.stack(
            [at] + [(at // d) % 64 for d in (48, 1)][:case["axes"] - 1]).int().contiguous()
        return state
    state["q"] = torch.randn((total, hq, D), generator=g, device=DEV).to(
        torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
    if op == "weights" or case.get("weights"):
        # what some tokens before have left
        state["sums"] = 0.02 * torch.rand((case["batch"], hkv, state["cap"]), generator=g, device=DEV)
    return state


# ------------------------------------------------------------------------------------------------------- the passes


def _gather(pages, table, at):
    """[B, kv heads, n, 128] in 32 bits: the tokens `at` [B, n] of each sequence."""
    page = pages.shape[2]
    ids = table.gather(1, at // page).clamp(min=0).long()
    return pages[ids, :, at % page].transpose(1, 2).float()


def _softmax(s, seen):
    """In place, over the keys that `seen` marks; a row that sees none gets 0."""
    s.masked_fill_(~seen, -math.inf)
    s.sub_(s.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    return s.div_(s.sum(-1, keepdim=True).clamp(min=1e-30))


def _norm_rope(x, w, cos, sin, cast):
    """x [rows, heads, D] in 32 bits."""
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    y = y.bfloat16().float() * w.float() if cast else y * w.float()
    y = y.bfloat16().float() if cast else y
    a, b = y[..., :D // 2], y[..., D // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _slots(s):
    """Of every packed row: its sequence, its slot in it, and the (page, slot in the page)."""
    cu, t = s["cu"].long(), torch.arange(sum(s["n_rows"]), device=DEV)
    b = torch.bucketize(t, cu[1:], right=True)
    at = s["lens"].long()[b] - cu[b + 1] + t
    return b, at, s["table"].long()[b, at // s["page"]], at % s["page"]


def _plain_rows(s):
    hq, hkv = s["hq"], s["hkv"]
    b, at, page, slot = _slots(s)
    pos = at[None] if s["positions"] is None else s["positions"].long()
    i = torch.arange(D // 2, device=DEV)
    angle = s["angles"][pos[torch.tensor(s["axis_of"], device=DEV)].T, i]
    cos, sin = angle[..., None, :, 0], angle[..., None, :, 1]
    x = s["x"].float().view(-1, hq + 2 * hkv, D)
    q = _norm_rope(x[:, :hq], s["q_norm"], cos, sin, s["cast"])
    k = _norm_rope(x[:, hq:hq + hkv], s["k_norm"], cos, sin, s["cast"])
    s["k"][page, :, slot] = k.bfloat16()
    s["v"][page, :, slot] = x[:, hq + hkv:].bfloat16()
    return q.to(torch.bfloat16 if s["dst"] == "bf16" else torch.float32)


def _prompt_rows(s, most):
    """Of the last `most` rows of each sequence (0: all), padded to as many: their packed places, whether they are
    there, and the keys that they see, [B, rows, keys]."""
    cu, lens = s["cu"].long(), s["lens"].long()
    n = min(most or s["max_rows"], s["max_rows"])
    i = torch.arange(n, device=DEV) - n
    there = i >= (cu[:-1] - cu[1:])[:, None]
    last = lens[:, None] + i
    key = torch.arange(s["max_len"], device=DEV)
    seen = (key <= last[..., None]) & ((key > last[..., None] - s["window"]) | (key < s["sinks"]))
    return (cu[1:, None] + i).clamp(min=0), there, seen & there[..., None]


def _scores(s, at, key):
    B, n = at.shape
    q = s["q"][at].float().view(B, n, s["hkv"], -1, D).permute(0, 2, 3, 1, 4)
    k = _gather(s["k"], s["table"], key)
    return torch.matmul(q, k[:, :, None].transpose(-1, -2)).mul_(SCALE)


def _plain_prompt(s):
    at, there, seen = _prompt_rows(s, 0)
    key = torch.arange(s["max_len"], device=DEV).expand(s["batch"], -1)
    p = _softmax(_scores(s, at, key), seen[:, None, None])
    o = torch.matmul(p, _gather(s["v"], s["table"], key)[:, :, None]).permute(0, 3, 1, 2, 4)
    out = torch.zeros_like(s["q"])
    out[at[there]] = o.reshape(*at.shape, s["hq"], D)[there].to(out.dtype)
    return out


def _plain_weights(s):
    at, there, seen = _prompt_rows(s, s["last"])
    key = torch.arange(s["max_len"], device=DEV).expand(s["batch"], -1)
    p = _softmax(_scores(s, at, key), seen[:, None, None])
    s["sums"][..., :s["max_len"]] += p.sum((2, 3))
    return s["sums"]


def _plain_decode(s):
    lens, B = s["lens"].long(), s["batch"]
    n = min(s["max_len"], s["window"] + s["sinks"])
    i = torch.arange(n, device=DEV).expand(B, n)
    past = (lens - n)[:, None].clamp(min=0)
    key = torch.where(i < min(n, s["sinks"]), i, i + past)
    seen = key < lens[:, None]
    key = torch.where(seen, key, 0)
    p = _softmax(_scores(s, torch.arange(B, device=DEV)[:, None], key), seen[:, None, None, None])
    o = torch.matmul(p, _gather(s["v"], s["table"], key)[:, :, None]).reshape(B, s["hq"], D).to(s["q"].dtype)
    if not s["weights"]:
        return o
    s["sums"].scatter_add_(2, key[:, None].expand(-1, s["hkv"], -1), p.sum((2, 3)))
    return o, s["sums"]


def _plain_evict(s):
    table, lens, refs, w, page = s["table"], s["lens"], s["refs"], s["weights_now"], s["page"]
    L, B, H, cap = w.shape
    cut = torch.minimum(s["keep"], lens)
    key = torch.arange(cap, device=DEV)
    always = (key < s["sinks"]) | (key >= (lens - s["recent"])[:, None])
    rank = torch.where(always[:, None], math.inf, w).masked_fill_(key >= lens[:, None, None], -math.inf)
    order = rank.sort(dim=-1, descending=True, stable=True)[1]
    chosen = torch.zeros_like(w, dtype=torch.bool).scatter_(-1, order, (key < cut[:, None, None]).expand_as(order))
    src = (~chosen).to(torch.int8).sort(dim=-1, stable=True)[1]
    fresh = key < cut[:, None, None]
    w.copy_(torch.where(fresh, w.gather(-1, src), 0.0))
    layer, b, h, to = torch.nonzero(fresh.expand_as(w), as_tuple=True)
    at = src[layer, b, h, to]
    ids = table.long()
    for x in (s["k"], s["v"]):
        x[layer, ids[b, to // page], h, to % page] = x[layer, ids[b, at // page], h, at % page]
    gone = (torch.arange(table.shape[1], device=DEV) >= ((cut + page - 1) // page)[:, None]) & (table >= 0)
    refs.index_add_(0, table.clamp(min=0).flatten().long(), -gone.int().flatten())
    table.masked_fill_(gone, -1)
    lens.copy_(cut)


def run(state):
    s, op = state, state["op"]
    if op == "evict":
        s["meta"].copy_(s["first"])
        s["weights_now"].copy_(s["first_weights"])
    if own:
        return _own(s)
    if op == "rows":
        return _plain_rows(s), s["k"], s["v"]
    if op == "prompt":
        return _plain_prompt(s)
    if op == "weights":
        return _plain_weights(s)
    if op == "decode":
        return _plain_decode(s)
    _plain_evict(s)
    return s["table"], s["lens"], s["refs"], s["weights_now"], s["k"], s["v"]


def _own(s):
    from transformer_decode_step_weight_gb300 import api

    op = s["op"]
    if op == "rows":
        q = api.qk_norm_rope(s["x"], s["q_norm"], s["k_norm"], s["angles"], s["k"], s["v"], s["table"], s["cu"], s["lens"],
                             EPS, positions=s["positions"], axes=s["axis_of"], cast=s["cast"],
                             dtype=torch.bfloat16 if s["dst"] == "bf16" else torch.float32)
        return q, s["k"], s["v"]
    if op == "prompt":
        if "work" not in s:
            s["work"] = torch.zeros(api.attn_prompt_workspace_bytes(), dtype=torch.uint8, device=DEV)
        return api.attn_prompt_window(s["q"], s["k"], s["v"], s["table"], s["cu"], s["lens"], SCALE, s["window"],
                                      n_sinks=s["sinks"], workspace=s["work"])
    if op == "weights":
        if "work" not in s:
            s["work"] = torch.zeros(api.attn_key_weights_workspace_bytes(s["batch"], sum(s["n_rows"]), s["hq"], s["hkv"],
                                                                         s["last"]), dtype=torch.uint8, device=DEV)
        api.attn_key_weights(s["q"], s["k"], s["table"], s["cu"], s["lens"], SCALE, s["sums"], last=s["last"],
                             window=s["window"], n_sinks=s["sinks"], workspace=s["work"])
        return s["sums"]
    if op == "decode":
        if "work" not in s:
            s["work"] = torch.zeros(api.attn_decode_window_workspace_bytes(s["batch"], s["hq"], s["hkv"],
                                                                           s["cap"] if s["weights"] else 0),
                                    dtype=torch.uint8, device=DEV)
        out = api.attn_decode_window(s["q"], s["k"], s["v"], s["table"], s["lens"], SCALE, s["window"],
                                     n_sinks=s["sinks"], key_weights=s.get("sums"), workspace=s["work"])
        return (out, s["sums"]) if s["weights"] else out
    if "cache" not in s:
        s["cache"] = api.PageCache(list(s["k"]), list(s["v"]), s["table"], s["lens"], s["refs"])
    s["cache"].evict(s["weights_now"], s["keep"], n_sinks=s["sinks"], n_recent=s["recent"])
    return s["table"], s["lens"], s["refs"], s["weights_now"], s["k"], s["v"]


# ------------------------------------------------------------------------------------------------- work and exact


def _seen(p, window, sinks):
    """Keys that the row at slot p sees."""
    return p + 1 if p < window else window + min(sinks, p + 1 - window)


def work(case):
    op, hkv = case["op"], case["hkv"]
    rows, lens = _lens(case)
    if op == "evict":
        moved = sum(max(0, min(case["keep"], n) - case["sinks"]) for n in lens if n > case["keep"])
        kept = sum(min(case["keep"], n) for n in lens)
        return {"bytes": case["layers"] * hkv * (moved * 4 * D * 2 + (sum(lens) + kept) * 4) + 8 * sum(lens),
                "flops": case["layers"] * hkv * sum(lens)}
    hq, total = case["hq"], sum(rows)
    if op == "rows":
        size = {"f32": 4, "bf16": 2}
        return {"bytes": total * D * ((hq + 2 * hkv) * size[case["src"]] + hq * size[case["dst"]] + 2 * hkv * 2 + 4),
                "flops": 8 * total * (hq + hkv) * D}
    size = 2 if case["dtype"] == "bf16" else 4
    last = case.get("last", 0)
    used = [min(n, last) if last else n for n in rows]
    seen = sum(_seen(p, case["window"], case["sinks"]) for n, m in zip(used, lens) for p in range(m - n, m))
    keys = sum(min(m, min(m, n - 1 + case["window"]) + case["sinks"]) for n, m in zip(used, lens) if n)
    if op == "weights":
        return {"bytes": keys * hkv * (D * 2 + 8) + sum(used) * hq * D * size, "flops": 2 * D * hq * seen}
    extra = 8 * hkv * keys if case.get("weights") else 0
    return {"bytes": keys * 2 * hkv * D * 2 + 2 * total * hq * D * size + extra, "flops": 4 * D * hq * seen}


def _exact_attend(s, b, rows, lasts):
    """(out [rows, hq, D], weights summed over the rows and a kv head's q heads [hkv, keys]) of the rows of sequence b
    whose last keys are `lasts`, in 64 bits."""
    hq, hkv, page, keys = s["hq"], s["hkv"], s["page"], int(s["lens"][b])
    where = torch.arange(keys, device=DEV)
    ids, slots = s["table"][b].long()[where // page], where % page
    far = lasts[:, None] - where
    hidden = (far < 0) | ((far >= s["window"]) & (where >= s["sinks"]))
    out = torch.zeros((len(rows), hq, D), dtype=torch.float64, device=DEV)
    sums = torch.zeros((hkv, keys), dtype=torch.float64, device=DEV)
    for h in range(hq):
        kv = h // (hq // hkv)
        w = (s["q"][rows, h].double() @ s["k"][ids, kv, slots].double().T / math.sqrt(D)).masked_fill(hidden, -math.inf)
        w = torch.softmax(w, -1)
        out[:, h] = w @ s["v"][ids, kv, slots].double()
        sums[kv] += w.sum(0)
    return out, sums


def _exact_rows(s):
    hq, hkv, page = s["hq"], s["hkv"], s["page"]
    cu, x = s["cu"].tolist(), s["x"].double().view(-1, hq + 2 * hkv, D)
    axis = torch.tensor(s["axis_of"], device=DEV)
    out = torch.zeros((x.shape[0], hq, D), dtype=torch.float64, device=DEV)

    def half(v):
        return v.bfloat16().double() if s["cast"] else v

    for b, m in enumerate(s["lens"].tolist()):
        row = torch.arange(cu[b], cu[b + 1], device=DEV)
        slot = torch.arange(m - len(row), m, device=DEV)
        pos = slot.expand(1, -1) if s["positions"] is None else s["positions"][:, row].long()
        turn = torch.view_as_complex(s["angles"].double())[pos[axis], torch.arange(D // 2, device=DEV)[:, None]].T
        for h in range(hq + hkv):
            v = x[row, h]
            v = half(v / (v.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt())
            v = half(v * (s["q_norm"] if h < hq else s["k_norm"]).double())
            z = torch.complex(v[:, :D // 2], v[:, D // 2:]) * turn
            v = torch.cat([z.real, z.imag], 1)
            if h < hq:
                out[row, h] = v
            else:
                s["k"][s["table"][b].long()[slot // page], h - hq, slot % page] = v.bfloat16()
                s["v"][s["table"][b].long()[slot // page], h - hq, slot % page] = x[row, h + hkv].bfloat16()
    return out, s["k"], s["v"]


def _exact_evict(s):
    page, w = s["page"], s["weights_now"].cpu().numpy()
    table, lens, refs = (s[n].cpu().numpy().copy() for n in ("table", "lens", "refs"))
    new = np.zeros_like(w)
    for b, n in enumerate(lens.tolist()):
        cut = min(n, s["keep"][b].item())
        if cut == n:
            new[:, b, :, :n] = w[:, b, :, :n]
            continue
        ids = torch.from_numpy(table[b].astype(np.int64)).to(DEV)
        middle = np.arange(s["sinks"], n - s["recent"])
        for l in range(w.shape[0]):
            for h in range(w.shape[2]):
                kept = np.ones(n, dtype=bool)
                kept[middle[np.lexsort((middle, -w[l, b, h, middle]))[cut - n + len(middle):]]] = False
                kept = np.nonzero(kept)[0]
                new[l, b, h, :cut] = w[l, b, h, kept]
                moved = kept != np.arange(cut)
                a, c = torch.from_numpy(kept[moved]).to(DEV), torch.from_numpy(np.arange(cut)[moved]).to(DEV)
                for x in (s["k"][l], s["v"][l]):
                    x[ids[c // page], h, c % page] = x[ids[a // page], h, a % page].clone()
        for i in range(-(-cut // page), -(-n // page)):
            refs[table[b, i]] -= 1
            table[b, i] = -1
        lens[b] = cut
    return table, lens, refs, new, s["k"], s["v"]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "rows":
        return _exact_rows(s)
    if op == "evict":
        return _exact_evict(s)
    cu, last = s["cu"].tolist(), case.get("last", 0)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    sums = s["sums"].double() if "sums" in s else None
    for b, n in enumerate(s["lens"].tolist()):
        rows = torch.arange(cu[b], cu[b + 1], device=DEV)
        rows = rows[-last:] if last else rows
        if len(rows):
            out[rows], add = _exact_attend(s, b, rows, torch.arange(n - len(rows), n, device=DEV))
            if sums is not None:
                sums[b, :, :n] += add
    return sums if op == "weights" else (out, sums) if sums is not None else out
