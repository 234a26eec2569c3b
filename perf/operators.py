"""Cases of the serving operators: page operations on the K/V cache, decode attention for sequences that share a
prefix, attention over packed prompts, and verification of drafted tokens by their probabilities.

Shapes are those of the Qwen3-8B (32 q heads, 8 kv heads, 36 layers, vocabulary 151936) and Qwen3-0.6B (16 q heads,
8 kv heads, 28 layers) configurations of this repository; caches are bf16 [pages, kv heads, page size, 128]. The plain
forms are elementary torch operations in 32 bits (64 for the sums of a drawn token, whose borders decide a whole
number); with `own` set, run() makes the framework's calls.
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


# ------------------------------------------------------------------------------------------------------ the cases


def listed():
    return [
        # several users' messages prefilled in one call: ragged, a few hundred tokens each
        dict(name="prompt-16-messages-bf16", op="prompt", dtype="bf16", hq=32, hkv=8, page=16, batch=16, rows_lo=20,
             rows_hi=700, past_hi=0, lens=1),
        # one long document from an empty cache: the largest, compute-bound
        dict(name="prompt-8192-bf16", op="prompt", dtype="bf16", hq=32, hkv=8, page=64, batch=1, rows_lo=8192,
             rows_hi=8192, past_hi=0, lens=2),
        # the next chunk of three conversations behind long caches, in the framework's own f32 rows; odd sizes
        dict(name="prompt-3-chunks-f32", op="prompt", dtype="f32", hq=16, hkv=8, page=16, batch=3, rows_lo=33,
             rows_hi=333, past_hi=12001, lens=3),
        # 64 samples of one 4096-token prompt, a few hundred tokens in; f32 as the decode step's q
        dict(name="shared-64x4096-f32", op="shared", dtype="f32", hq=32, hkv=8, page=16, groups=1, batch=64,
             shared=4096, tail_hi=512, lens=4),
        # 64 answers over one 32768-token document
        dict(name="shared-64x32768-bf16", op="shared", dtype="bf16", hq=32, hkv=8, page=16, groups=1, batch=64,
             shared=32768, tail_hi=512, lens=5),
        # eight prompts with their own samples each
        dict(name="shared-8-groups-f32", op="shared", dtype="f32", hq=32, hkv=8, page=16, groups=8, batch=48,
             shared=1900, tail_hi=300, lens=6),
        # four samples of a short prompt: latency
        dict(name="shared-4x300-f32", op="shared", dtype="f32", hq=16, hkv=8, page=16, groups=1, batch=4, shared=300,
             tail_hi=40, lens=7),
        # a prompt forked to 63 samples, each then given room for its next token: one partial page copied per sample
        dict(name="pages-fork-63", op="fork", layers=36, hkv=8, page=16, pages=1024, parent=4101, n=63, lens=8),
        # a cache of the small model defragmented after half of its sequences ended
        dict(name="pages-compact", op="compact", layers=28, hkv=8, page=16, pages=1200, n=40, len_hi=420, lens=9),
        # two pages copied: latency
        dict(name="pages-copy-2", op="copy", layers=36, hkv=8, page=16, pages=64, n=2, lens=10),
        # one sequence's drafts checked: latency
        dict(name="verify-1x4", op="verify", batch=1, k=4, vocab=151936, lens=11),
        # a whole batch with 4 drafts each
        dict(name="verify-64x5", op="verify", batch=64, k=5, vocab=151936, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "shared", "shared", "fork", "compact", "copy", "verify", "verify"])
    seed = rng.randrange(1 << 30)
    hq, hkv = rng.choice([(32, 8), (16, 8), (8, 8), (16, 2), (4, 2)])
    page = rng.choice([16, 16, 32, 64, 128, 24, 7])
    if op == "prompt":
        batch = _log(rng, 1, 16)
        hi = _log(rng, 1, 4096 // batch + 40)
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), hq=hq, hkv=hkv, page=page, batch=batch,
                    rows_lo=rng.choice([0, 1, (hi + 1) // 2]), rows_hi=hi, past_hi=rng.choice([0, _log(rng, 1, 8000)]),
                    lens=seed)
    if op == "shared":
        groups = _log(rng, 1, 8)
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), hq=hq, hkv=hkv, page=page, groups=groups,
                    batch=groups + _log(rng, 1, 56), shared=_log(rng, 16, 20000 // groups), tail_hi=_log(rng, 1, 600),
                    lens=seed)
    if op != "verify":
        pages = 12800 // page
        case = dict(op=op, layers=rng.randint(1, 36), hkv=hkv, page=page, pages=pages, lens=seed)
        if op == "fork":
            return dict(case, parent=_log(rng, 1, pages // 3 * page), n=_log(rng, 1, min(100, pages // 4)))
        if op == "compact":
            return dict(case, n=rng.randint(2, 30), len_hi=_log(rng, 1, 640))
        return dict(case, n=_log(rng, 1, min(200, pages // 2)))
    return dict(op=op, batch=_log(rng, 1, 64), k=rng.randint(1, 8), vocab=_log(rng, 50, 151936), lens=seed)


def _lens(case):
    """The lengths of a case's sequences, from the case alone."""
    r = random.Random(case["lens"])
    if case["op"] == "prompt":
        rows = [r.randint(case["rows_lo"], case["rows_hi"]) for _ in range(case["batch"])]
        rows[-1] = max(rows[-1], 1)
        past = [r.randint(case["past_hi"] // 2, case["past_hi"]) for _ in rows]
        return rows, [n + p for n, p in zip(rows, past)]
    if case["op"] == "shared":
        cuts = sorted(r.sample(range(1, case["batch"]), case["groups"] - 1))
        cu = [0] + cuts + [case["batch"]]
        shared = [r.randint((case["shared"] + 1) // 2, case["shared"]) if case["groups"] > 1 else case["shared"]
                  for _ in range(case["groups"])]
        tails = [r.randint(0, case["tail_hi"]) for _ in range(case["batch"])]
        return cu, shared, tails
    if case["op"] == "compact":
        room, lens = case["pages"], []
        for _ in range(case["n"]):
            n = min(r.randint(1, case["len_hi"]), room * case["page"])
            room -= -(-n // case["page"])
            lens.append(n)
        return lens
    return None


# ------------------------------------------------------------------------------------------------------ the inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _caches(g, *shape):
    # values as a filled cache has them, N(0, 1)
    k = torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    v = torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    return k, v


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _table(rows, width, n_pages, r):
    """Page table of the sequences whose logical pages `rows` names (numbers of pages, shared ones repeated)."""
    perm = list(range(n_pages))
    r.shuffle(perm)
    return _ints([[perm[p] for p in row] + [-1] * (width - len(row)) for row in rows])


def prepare(case, seed):
    g, r, op = _gen(seed), random.Random(seed), case["op"]
    state = dict(case)
    if op in ("prompt", "shared"):
        page, hkv = case["page"], case["hkv"]
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        rows, used = [], 0
        if op == "prompt":
            n_rows, lens = _lens(case)
            for n in lens:
                need = -(-n // page)
                rows.append(list(range(used, used + need)))
                used += need
            total = sum(n_rows)
            state["cu"] = _ints(np.concatenate([[0], np.cumsum(n_rows)]).tolist())
            state["max_rows"] = max(n_rows)
        else:
            cu, shared, tails = _lens(case)
            lens = []
            for i, n in enumerate(shared):
                # whole pages of the prefix are shared; its partly filled last page each sequence has for itself
                head = list(range(used, used + n // page))
                used += len(head)
                for b in range(cu[i], cu[i + 1]):
                    lens.append(n + tails[b])
                    need = -(-lens[-1] // page) - len(head)
                    rows.append(head + list(range(used, used + need)))
                    used += need
            total = case["batch"]
            state["cu"] = _ints(cu)
            state["shared_lens"] = _ints([n // page * page for n in shared])
        state["max_len"] = max(lens)
        state["lens"] = _ints(lens)
        state["table"] = _table(rows, max(max(len(x) for x in rows), 1), used + 3, r)
        state["k"], state["v"] = _caches(g, used + 3, hkv, page, D)
        state["q"] = torch.randn((total, case["hq"], D), generator=g, device=DEV).to(dtype)
        return state
    if op == "verify":
        B, k, V = case["batch"], case["k"], case["vocab"]
        # the draft model's distribution and a target near it, so that most drafts are accepted
        z = torch.randn((B, k, V), generator=g, device=DEV) * 2.5
        state["p"] = torch.softmax(z + 0.4 * torch.randn((B, k, V), generator=g, device=DEV), -1)
        state["d"] = torch.softmax(z[:, :k - 1], -1).contiguous()
        pick = torch.rand((B, k - 1, 1), generator=g, device=DEV)
        # one drafted token each, drawn from the draft model
        state["draft"] = ((state["d"].cumsum(-1) <= pick).sum(-1).clamp(max=V - 1)).to(torch.int32)
        state["u"] = torch.rand((B, k), generator=g, device=DEV)
        state["tok"] = torch.zeros(B, dtype=torch.int32, device=DEV)
        state["start"] = _ints([[r.randrange(4000), r.randrange(8)] for _ in range(B)])
        state["pos"], state["step"] = state["start"][:, 0].clone(), state["start"][:, 1].clone()
        state["max_steps"] = 16
        state["out_tokens"] = torch.full((B, 16), -1, dtype=torch.int32, device=DEV)
        return state
    # page operations: every layer's cache in one tensor; the table, lengths and reference counts in another, so
    # that a pass can start from the same ones
    L, hkv, page, P, n = case["layers"], case["hkv"], case["page"], case["pages"], case["n"]
    state["k"], state["v"] = _caches(g, L, P, hkv, page, D)
    if op == "copy":
        ids = list(range(P))
        r.shuffle(ids)
        state["src"], state["dst"] = _ints(ids[:n]), _ints(ids[n:2 * n])
        return state
    if op == "fork":
        seqs, lens = n + 1, [case["parent"]] + [0] * n
        state["parents"], state["children"] = _ints([0] * n), _ints(list(range(1, n + 1)))
        state["grow"] = _ints([1] * seqs)
    else:
        lens = _lens(case)
        seqs = n
        state["cut"] = _ints([0 if i % 2 else -1 for i in range(n)])
    width = max(-(-(m + 1) // page) for m in lens)
    rows, used = [], 0
    for m in lens:
        need = -(-m // page)
        rows.append(list(range(used, used + need)))
        used += need
    table = _table(rows, width, P, r)
    refs = torch.zeros(P, dtype=torch.int32, device=DEV)
    refs[table[table >= 0].long()] = 1
    state["first"] = torch.cat([table.flatten(), _ints(lens), refs])
    state["meta"] = state["first"].clone()
    state["table"] = state["meta"][:seqs * width].view(seqs, width)
    state["lens"] = state["meta"][seqs * width:seqs * width + seqs]
    state["refs"] = state["meta"][seqs * width + seqs:]
    return state


# ------------------------------------------------------------------------------------------------------- the passes


def _gather(pages, table, n):
    """[B, kv heads, n, 128] in 32 bits: the first n tokens of each sequence."""
    width = -(-n // pages.shape[2])
    x = pages[table[:, :width].clamp(min=0).long()]
    return x.transpose(1, 2).reshape(table.shape[0], pages.shape[1], -1, D)[:, :, :n].float()


def _attend(q, k, v, seen):
    """softmax(scale q k^T) v over the keys that `seen` [B, 1, 1, n, keys] marks; a row that sees none gives 0."""
    s = torch.matmul(q, k.transpose(-1, -2)) * SCALE
    s.masked_fill_(~seen, -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    s.sub_(m).exp_()
    return torch.matmul(s, v) / s.sum(-1, keepdim=True).clamp(min=1e-30)


def _plain_prompt(s):
    q, cu, lens = s["q"], s["cu"].long(), s["lens"].long()
    B, hq, hkv, n, keys = s["batch"], s["hq"], s["hkv"], s["max_rows"], s["max_len"]
    rows = cu[1:] - cu[:-1]
    i = torch.arange(n, device=DEV)
    at = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)
    qp = q[at].float().view(B, n, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4)
    last = lens[:, None] - rows[:, None] + i
    seen = (torch.arange(keys, device=DEV) <= last[..., None])[:, None, None]
    o = _attend(qp, _gather(s["k"], s["table"], keys)[:, :, None], _gather(s["v"], s["table"], keys)[:, :, None], seen)
    o = o.permute(0, 3, 1, 2, 4).reshape(B * n, hq, D)
    t = torch.arange(q.shape[0], device=DEV)
    b = torch.bucketize(t, cu[1:], right=True)
    return o[b * n + t - cu[b]].to(q.dtype)


def _plain_shared(s):
    q, hq, hkv, n = s["q"], s["hq"], s["hkv"], s["max_len"]
    qp = q.float().view(q.shape[0], hkv, hq // hkv, 1, D)
    seen = (torch.arange(n, device=DEV) < s["lens"][:, None])[:, None, None, None]
    o = _attend(qp, _gather(s["k"], s["table"], n)[:, :, None], _gather(s["v"], s["table"], n)[:, :, None], seen)
    return o.reshape(q.shape[0], hq, D).to(q.dtype)


def _plain_copy(s, src, dst):
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]


def _plain_fork(s):
    rows = s["table"][s["parents"].long()]
    s["table"][s["children"].long()] = rows
    s["lens"][s["children"].long()] = s["lens"][s["parents"].long()]
    s["refs"].index_add_(0, rows.clamp(min=0).flatten().long(), (rows >= 0).int().flatten())


def _plain_extend(s):
    table, lens, refs, page = s["table"], s["lens"], s["refs"], s["page"]
    had, has = (lens + page - 1) // page, (lens + s["grow"] + page - 1) // page
    last = table.gather(1, (had - 1).clamp(min=0).long()[:, None])[:, 0].long().clamp(min=0)
    partial = (lens % page != 0) & (s["grow"] > 0) & (refs[last] > 1)
    before = ((last[:, None] == last) & partial & partial[:, None]).tril(-1).sum(1)
    own_page = partial & (refs[last] - before > 1)
    need = has - had + own_page
    at = need.cumsum(0) - need
    free = torch.nonzero(refs == 0)[:, 0].int()
    i = torch.arange(table.shape[1], device=DEV)
    fresh = (i >= (had - own_page.int())[:, None]) & (i < has[:, None])
    rank = (at + own_page.int() - had)[:, None] + i
    new = free[rank.clamp(0, free.numel() - 1)]
    _plain_copy(s, last[own_page], new.gather(1, (had - 1).clamp(min=0).long()[:, None])[:, 0][own_page].long())
    refs.index_add_(0, last, -own_page.int())
    table.copy_(torch.where(fresh, new, table))
    refs.index_add_(0, table.clamp(min=0).flatten().long(), fresh.int().flatten())
    lens.add_(s["grow"])


def _plain_trim(s):
    table, lens, refs, page = s["table"], s["lens"], s["refs"], s["page"]
    n = torch.where(s["cut"] >= 0, torch.minimum(s["cut"], lens), lens)
    gone = (torch.arange(table.shape[1], device=DEV) >= ((n + page - 1) // page)[:, None]) & (table >= 0)
    refs.index_add_(0, table.clamp(min=0).flatten().long(), -gone.int().flatten())
    table.masked_fill_(gone, -1)
    lens.copy_(n)


def _plain_compact(s):
    table, refs = s["table"], s["refs"]
    ids = torch.arange(refs.numel(), device=DEV)
    live = refs > 0
    n = live.sum()
    src, dst = torch.nonzero(live & (ids >= n))[:, 0], torch.nonzero(~live & (ids < n))[:, 0]
    _plain_copy(s, src, dst)
    to = ids.clone()
    to[src] = dst
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table))
    refs[dst] = refs[src]
    refs[src] = 0
    return n.int().view(1)


def _plain_verify(s):
    p, d, draft, u, k = s["p"], s["d"], s["draft"].long(), s["u"], s["k"]
    B = p.shape[0]
    b = torch.arange(B, device=DEV)
    pd = p[:, :k - 1].gather(2, draft[..., None])[..., 0].double()
    qd = d.gather(2, draft[..., None])[..., 0].double()
    ok = u[:, :k - 1].double() * qd < pd
    m = ok.int().cumprod(1).sum(1)
    row = p[b, m].double()
    if k > 1:
        less = d[b, m.clamp(max=k - 2)].double() * (m < k - 1)[:, None]
        rest = (row - less).clamp(min=0)
        row = torch.where(rest.sum(1, keepdim=True) > 0, rest, row)
    c = row.cumsum(1)
    t = (c <= u[:, k - 1:].double() * c[:, -1:]).sum(1).clamp(max=p.shape[2] - 1)
    i = torch.arange(k, device=DEV)
    new = torch.where(i == m[:, None], t[:, None], torch.nn.functional.pad(draft, (0, 1)))
    at = s["step"][:, None].long() + i
    rows = torch.full_like(s["out_tokens"], -1)
    rows.scatter_(1, at, torch.where(i <= m[:, None], new, -1).int())
    s["out_tokens"].copy_(rows)
    s["tok"].copy_(t)
    s["pos"].add_(m + 1)
    s["step"].add_(m + 1)
    return m.int()


def run(state):
    s, op = state, state["op"]
    if op in ("fork", "compact"):
        s["meta"].copy_(s["first"])
    elif op == "verify":
        s["pos"].copy_(s["start"][:, 0])
        s["step"].copy_(s["start"][:, 1])
        s["out_tokens"].fill_(-1)
    if own:
        return _own(s)
    if op == "prompt":
        return _plain_prompt(s)
    if op == "shared":
        return _plain_shared(s)
    if op == "copy":
        _plain_copy(s, s["src"].long(), s["dst"].long())
        return s["k"], s["v"]
    if op == "fork":
        _plain_fork(s)
        _plain_extend(s)
        return s["table"], s["lens"], s["refs"], s["k"], s["v"]
    if op == "compact":
        _plain_trim(s)
        n = _plain_compact(s)
        return s["table"], s["lens"], s["refs"], n, s["k"], s["v"]
    m = _plain_verify(s)
    return m, s["out_tokens"], s["tok"], s["pos"], s["step"]


def _own(s):
    from transformer_decode_step_weight_gb300 import api

    op = s["op"]
    if op == "prompt":
        if "work" not in s:
            s["work"] = torch.zeros(api.attn_prompt_workspace_bytes(), dtype=torch.uint8, device=DEV)
        return api.attn_prompt(s["q"], s["k"], s["v"], s["table"], s["cu"], s["lens"], SCALE, workspace=s["work"])
    if op == "shared":
        if "work" not in s:
            s["work"] = torch.zeros(api.attn_shared_workspace_bytes(s["batch"], s["hq"], s["hkv"]), dtype=torch.uint8,
                                    device=DEV)
        return api.attn_decode_shared(s["q"], s["k"], s["v"], s["table"], s["lens"], s["cu"], s["shared_lens"], SCALE,
                                      workspace=s["work"])
    if op == "verify":
        if "work" not in s:
            s["work"] = torch.zeros(api.verify_sample_workspace_bytes(s["batch"]), dtype=torch.uint8, device=DEV)
        m = api.verify_sample(s["p"], s["d"], s["draft"], s["u"], s["tok"], s["pos"], s["step"], s["out_tokens"],
                              workspace=s["work"])
        return m, s["out_tokens"], s["tok"], s["pos"], s["step"]
    if "cache" not in s:
        s["cache"] = api.PageCache(list(s["k"]), list(s["v"]), s.get("table"), s.get("lens"), s.get("refs"))
    c = s["cache"]
    if op == "copy":
        c.copy(s["src"], s["dst"])
        return s["k"], s["v"]
    if op == "fork":
        c.fork(s["parents"], s["children"])
        c.extend(s["grow"])
        return s["table"], s["lens"], s["refs"], s["k"], s["v"]
    c.trim(s["cut"])
    n = c.compact()
    return s["table"], s["lens"], s["refs"], n, s["k"], s["v"]


# ------------------------------------------------------------------------------------------------- work and exact


def work(case):
    op = case["op"]
    if op in ("prompt", "shared"):
        size = 2 if case["dtype"] == "bf16" else 4
        token = 2 * case["hkv"] * D * 2
        if op == "prompt":
            rows, lens = _lens(case)
            seen = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(rows, lens))
            keys, total = sum(m for n, m in zip(rows, lens) if n), sum(rows)
        else:
            cu, shared, tails = _lens(case)
            whole = [n // case["page"] * case["page"] for n in shared]
            keys = sum(whole) + sum(tails) + sum((n - w) * (b - a) for n, w, a, b in zip(shared, whole, cu, cu[1:]))
            seen = sum(n * (b - a) for n, a, b in zip(shared, cu, cu[1:])) + sum(tails)
            total = case["batch"]
        return {"bytes": keys * token + 2 * total * case["hq"] * D * size, "flops": 4 * D * case["hq"] * seen}
    if op == "verify":
        return {"bytes": case["batch"] * case["vocab"] * 4 * (2 if case["k"] > 1 else 1),
                "flops": 3 * case["batch"] * case["vocab"]}
    one = case["layers"] * 2 * case["hkv"] * case["page"] * D * 2
    if op == "copy":
        return {"bytes": 2 * case["n"] * one, "flops": 0}
    page = case["page"]
    if op == "fork":
        entries = case["n"] * -(-case["parent"] // page)
        copies = case["n"] if case["parent"] % page else 0
        return {"bytes": (copies + (1 if copies else 0)) * one + 8 * entries + 4 * case["pages"], "flops": 0}
    lens = _lens(case)
    need = [-(-n // page) for n in lens]
    live = sum(need[0::2])
    # the live pages lie anywhere: the share of them past the first `live` ids moves
    moved = max(1, live * (case["pages"] - live) // case["pages"])
    return {"bytes": 2 * moved * one + 4 * (2 * case["pages"] + sum(need)), "flops": 0}


def _exact_rows(s, b, rows, lasts, keys):
    """Attention in 64 bits of the query rows `rows` of sequence b; row i sees the keys 0 .. lasts[i]."""
    hq, hkv, page = s["hq"], s["hkv"], s["page"]
    where = torch.arange(keys, device=DEV)
    ids, slots = s["table"][b].long()[where // page], where % page
    k, v = s["k"][ids, :, slots].double(), s["v"][ids, :, slots].double()
    out = torch.zeros((len(rows), hq, D), dtype=torch.float64, device=DEV)
    for h in range(hq):
        w = s["q"][rows, h].double() @ k[:, h // (hq // hkv)].T / math.sqrt(D)
        w = torch.where(where <= lasts[:, None], w, torch.full_like(w, -math.inf))
        some = lasts >= 0
        out[some, h] = torch.softmax(w[some], -1) @ v[:, h // (hq // hkv)]
    return out


def _exact_pages(s):
    """The page operations one by one on the host: (table, lengths, counts, (from, to) of each copied page, n)."""
    page, first = s["page"], s["first"].cpu().numpy()
    seqs, width = s["table"].shape
    table = [[int(p) for p in row if p >= 0] for row in first[:seqs * width].reshape(seqs, width)]
    lens = [int(n) for n in first[seqs * width:seqs * width + seqs]]
    refs = [int(n) for n in first[seqs * width + seqs:]]
    moves, live = [], None
    if s["op"] == "fork":
        for a, c in zip(s["parents"].tolist(), s["children"].tolist()):
            table[c], lens[c] = list(table[a]), lens[a]
            for p in table[a]:
                refs[p] += 1
        empty = [p for p, n in enumerate(refs) if n == 0]
        for q, n in enumerate(s["grow"].tolist()):
            if n > 0 and lens[q] % page and refs[table[q][-1]] > 1:
                to = empty.pop(0)
                moves.append((table[q][-1], to))
                refs[table[q][-1]] -= 1
                refs[to] = 1
                table[q][-1] = to
            lens[q] += n
            while len(table[q]) * page < lens[q]:
                to = empty.pop(0)
                refs[to] = 1
                table[q].append(to)
    else:
        for q, n in enumerate(s["cut"].tolist()):
            if 0 <= n < lens[q]:
                while (len(table[q]) - 1) * page >= n and table[q]:
                    refs[table[q].pop()] -= 1
                lens[q] = n
        live = sum(n > 0 for n in refs)
        holes = [p for p in range(live) if refs[p] == 0]
        new = {}
        for p in range(live, len(refs)):
            if refs[p] > 0:
                new[p] = holes.pop(0)
                moves.append((p, new[p]))
                refs[new[p]], refs[p] = refs[p], 0
        table = [[new.get(p, p) for p in row] for row in table]
    table = np.array([row + [-1] * (width - len(row)) for row in table], dtype=np.int32).reshape(seqs, width)
    return table, np.array(lens, dtype=np.int32), np.array(refs, dtype=np.int32), moves, live


def _exact_verify(s):
    k, V = s["k"], s["vocab"]
    p, d, draft, u = (s[n].cpu().numpy().astype(np.float64) for n in ("p", "d", "draft", "u"))
    start = s["start"].cpu().numpy()
    B = p.shape[0]
    m, tok = np.zeros(B, np.int32), np.zeros(B, np.int32)
    rows = np.full((B, s["max_steps"]), -1, np.int32)
    for b in range(B):
        while m[b] < k - 1 and u[b, m[b]] * d[b, m[b], int(draft[b, m[b]])] < p[b, m[b], int(draft[b, m[b]])]:
            m[b] += 1
        mass = p[b, m[b]]
        if m[b] < k - 1:
            rest = np.maximum(mass - d[b, m[b]], 0)
            mass = rest if rest.sum() > 0 else mass
        steps = np.cumsum(mass)
        tok[b] = min(int(np.searchsorted(steps, u[b, k - 1] * steps[-1], side="right")), V - 1)
        line = [int(t) for t in draft[b, :m[b]]] + [int(tok[b])]
        rows[b, start[b, 1]:start[b, 1] + len(line)] = line
    add = (m + 1).astype(np.int32)
    return m, rows, tok, start[:, 0] + add, start[:, 1] + add


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "prompt":
        out, cu = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV), s["cu"].tolist()
        for b, n in enumerate(s["lens"].tolist()):
            rows = torch.arange(cu[b], cu[b + 1], device=DEV)
            if len(rows):
                out[rows] = _exact_rows(s, b, rows, torch.arange(n - len(rows), n, device=DEV), n)
        return out
    if op == "shared":
        return torch.cat([_exact_rows(s, b, torch.tensor([b], device=DEV), torch.tensor([n - 1], device=DEV), n)
                          for b, n in enumerate(s["lens"].tolist())])
    if op == "verify":
        return _exact_verify(s)
    k, v = s["k"], s["v"]
    if op == "copy":
        moves, head = list(zip(s["src"].tolist(), s["dst"].tolist())), ()
    else:
        table, lens, refs, moves, live = _exact_pages(s)
        head = (table, lens, refs) if live is None else (table, lens, refs, np.array([live], dtype=np.int32))
    for a, b in moves:
        k[:, b] = k[:, a].clone()
        v[:, b] = v[:, a].clone()
    return (*head, k, v)
