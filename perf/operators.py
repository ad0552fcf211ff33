"""The attention half of a decoder layer, operator by operator: cases, inputs, plain forms and exact values.

Four operators stand beside the mixture-of-experts layer of this package:

  map      block tables, positions and cache slots of the new tokens, from the requests' lengths (moe_kv_map)
  rope     per-head RMS norm of queries and keys and the position rotation, keys and values written into
           the paged cache (moe_qk_norm_rope)
  decode   attention of a window of up to 8 new tokens a request over the paged cache (moe_attn_decode)
  prefill  attention of a prompt chunk over the paged cache (moe_attn_prefill)

With `own` false, run() computes them with elementary torch operations in 32 bits; with `own` true it
makes the calls of a user's program.
"""
from __future__ import annotations

import math
import random

import torch

own = False

E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one verify window (a token and 4 drafts) of a single user at a 4K context
        {"name": "map_window", "op": "map", "B": 1, "q": 5, "kv": 4096, "page": 16, "pad": 3},
        # a batch of requests, one to eight tokens each, in a step captured with padding rows
        {"name": "map_batch", "op": "map", "B": 384, "q": 8, "kv": 32768, "page": 16, "pad": 100},
        # a verify window behind a 128K prompt, half rotation of the whole head, 8-bit cache
        {"name": "rope_window", "op": "rope", "T": 5, "heads": 16, "kv_heads": 2, "dim": 128, "rot": 128,
         "interleaved": False, "norm": True, "e4m3": True, "page": 64, "kv": 131072, "head_major": False},
        # a batch's tokens, interleaved rotation of half of a short head, without norms, head-major pages
        {"name": "rope_batch", "op": "rope", "T": 257, "heads": 32, "kv_heads": 8, "dim": 64, "rot": 32,
         "interleaved": True, "norm": False, "e4m3": False, "page": 16, "kv": 32768, "head_major": True},
        # a whole prompt chunk of the layer's width
        {"name": "rope_chunk", "op": "rope", "T": 8192, "heads": 16, "kv_heads": 2, "dim": 128, "rot": 128,
         "interleaved": False, "norm": True, "e4m3": False, "page": 64, "kv": 8192, "head_major": False},
        # the next token of a short chat
        {"name": "decode_token", "op": "decode", "B": 1, "q": 1, "kv": 997, "heads": 16, "kv_heads": 2, "dim": 128,
         "e4m3": False, "page": 16, "head_major": False, "window": 0, "softcap": 0.0, "slopes": False},
        # a verify window of one user behind a 128K prompt in the 8-bit cache
        {"name": "decode_window_128k", "op": "decode", "B": 1, "q": 5, "kv": 131072, "heads": 16, "kv_heads": 2,
         "dim": 128, "e4m3": True, "page": 64, "head_major": False, "window": 0, "softcap": 0.0, "slopes": False},
        # the largest: one token of each of 64 ragged requests
        {"name": "decode_batch", "op": "decode", "B": 64, "q": 1, "kv": 32768, "heads": 32, "kv_heads": 4, "dim": 64,
         "e4m3": False, "page": 16, "head_major": True, "window": 0, "softcap": 0.0, "slopes": False},
        # ragged windows of up to 5 tokens, 5 query heads to a cached one, capped scores in a sliding window
        {"name": "decode_capped", "op": "decode", "B": 24, "q": 5, "kv": 12000, "heads": 20, "kv_heads": 4, "dim": 128,
         "e4m3": False, "page": 32, "head_major": False, "window": 4096, "softcap": 30.0, "slopes": False},
        # a chunk of the layer's longest prompt piece, from the prompt's first token
        {"name": "prefill_chunk", "op": "prefill", "B": 1, "q": 8192, "kv": 8192, "heads": 16, "kv_heads": 2,
         "dim": 128, "e4m3": False, "page": 64, "head_major": False, "window": 0, "softcap": 0.0, "slopes": False,
         "prefix": 0},
        # a later chunk of a 64K prompt: most keys come from the cache
        {"name": "prefill_64k", "op": "prefill", "B": 1, "q": 2048, "kv": 65536, "heads": 16, "kv_heads": 2,
         "dim": 128, "e4m3": True, "page": 64, "head_major": False, "window": 0, "softcap": 0.0, "slopes": False,
         "prefix": 0},
        # several ragged prompts in one chunk, a bias by distance, and image tokens that see one another
        {"name": "prefill_packed", "op": "prefill", "B": 6, "q": 701, "kv": 1500, "heads": 12, "kv_heads": 4,
         "dim": 64, "e4m3": False, "page": 16, "head_major": True, "window": 0, "softcap": 0.0, "slopes": True,
         "prefix": 300},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["map", "rope", "decode", "decode", "prefill", "prefill"])
    page = rng.choice([1, 8, 16, 16, 32, 48, 64, 64, 128])
    if op == "map":
        return {"op": op, "B": _spread(rng, 1, 384), "q": rng.choice([1, 1, 5, 8]), "kv": _spread(rng, 1, 32768),
                "page": max(page, 8), "pad": rng.choice([0, 1, rng.randrange(200)])}
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 8]) if kv_heads < 8 else rng.choice([1, 2, 4])
    case = {"op": op, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": rng.choice([64, 128, 128]),
            "e4m3": rng.random() < 0.4, "page": page, "head_major": rng.random() < 0.4}
    if op == "rope":
        dim = case["dim"]
        width = (case["heads"] + 2 * kv_heads) * dim
        case |= {"T": _spread(rng, 1, min(8192, 8192 * 2560 // width)), "kv": _spread(rng, 8192, 262144),
                 "rot": rng.choice([dim, dim, dim // 2, dim // 4]), "interleaved": rng.random() < 0.4,
                 "norm": rng.random() < 0.7}
        return case
    case |= {"window": rng.choice([0, 0, 0, _spread(rng, 16, 4096)]), "softcap": rng.choice([0.0, 0.0, 30.0, 50.0]),
             "slopes": rng.random() < 0.2}
    if op == "decode":
        q = rng.choice([1, 1, 2, 5, 5, 8])
        room = 64 * 32768 * 4 * 64 // (kv_heads * case["dim"])  # cached tokens, as many bytes as the largest case's
        room = min(room, 64 * 32768 * 256 // (case["heads"] * q * 8))
        B = _spread(rng, 1, 96)
        return case | {"B": B, "q": q, "kv": _spread(rng, q, max(q, min(131072, room // B)))}
    q = _spread(rng, 9, 4096)
    B = min(rng.choice([1, 1, 1, 2, 3, 6]), 8192 // q)
    most = max(q, min(65536, 16 * 2048 * 65536 // (B * q * case["heads"])))
    return case | {"B": B, "q": q, "kv": _spread(rng, q, most), "prefix": rng.choice([0, 0, rng.randrange(1, q)])}


def _lengths(case):
    """(cached tokens before the step, new tokens) of each request: the case's own, the same for every seed."""
    r = random.Random("%d %d %d" % (case["B"], case["q"], case["kv"]))
    new, old = [], []
    for b in range(case["B"]):
        n = case["q"] if b == 0 or case["q"] == 1 else r.randint(max(1, case["q"] // 4), case["q"])
        total = case["kv"] if b == 0 else r.randint(min(case["kv"], max(n, case["kv"] // 8)), case["kv"])
        new.append(n)
        old.append(max(total, n) - n)
    return old, new


def _rows(case):
    """Per request: (lowest, one past the highest) visible key of each of its queries, as plain integers."""
    old, new = _lengths(case)
    out = []
    for o, n in zip(old, new):
        pre = min(case.get("prefix", 0), o + n)
        out.append([(max(0, o + i + 1 - case["window"]) if case["window"] else 0, max(o + i + 1, pre)) for i in range(n)])
    return out


def work(case):
    if case["op"] == "map":
        old, new = _lengths(case)
        T = sum(new) + case["pad"]
        p = case["page"]
        pages = sum(-(-(o + n) // p) - -(-o // p) for o, n in zip(old, new))
        # lengths in; lengths, offsets, positions and slots out; a page id read and written for each new page,
        # one read for each partly filled page that is gone on with
        return {"bytes": 8 * case["B"] + 4 * (2 * case["B"] + 1) + 8 * T + 8 * pages + 4 * case["B"] + 4, "flops": 0}
    D, Hq, Hk = case["dim"], case["heads"], case["kv_heads"]
    el = 1 if case["e4m3"] else 2
    if case["op"] == "rope":
        T = case["T"]
        by = T * (2 * (Hq + 2 * Hk) * D + 2 * Hq * D + 2 * Hk * D * el + 8) + case["rot"] // 2 * 4
        return {"bytes": by, "flops": T * (Hq + Hk) * (4 * D + 3 * case["rot"])}
    old, new = _lengths(case)
    keys = pairs = 0
    for rows in _rows(case):
        keys += max(h for _, h in rows) - min(l for l, _ in rows)
        pairs += sum(h - l for l, h in rows)
    by = keys * Hk * D * 2 * el + sum(new) * Hq * D * 4 + 4 * sum(-(-(o + n) // case["page"]) for o, n in zip(old, new))
    return {"bytes": by, "flops": 4 * D * Hq * pairs}


# ---------------------------------------------------------------- inputs

def _table(old, new, page, g, dev, spare):
    """A block table of distinct pages in random order for the tokens of `old` (and `new`), and the pages left over."""
    have = [-(-(o + n) // page) for o, n in zip(old, new)]
    width = max(have) + 2
    n_pages = sum(have) + spare
    ids = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    count = torch.tensor(have, device=dev)
    col = torch.arange(width, device=dev)
    used = col[None] < count[:, None]
    at = (torch.cumsum(count, 0) - count)[:, None] + col[None]
    table = torch.where(used, ids[at.clamp(max=n_pages - 1)], torch.full((), -1, dtype=torch.int32, device=dev))
    return table.contiguous(), ids[sum(have):].contiguous(), n_pages


def _cache(case, n_pages, g, dev, fill):
    """A paged cache [page, token, head, dim] of the case's type and order; stale values in every place."""
    shape = (n_pages, case["page"], case["kv_heads"], case["dim"])
    store = (n_pages, case["kv_heads"], case["page"], case["dim"]) if case["head_major"] else shape
    x = torch.empty(store, dtype=torch.bfloat16, device=dev)
    if fill:
        x.normal_(generator=g)
    else:
        x.zero_()
    if case["e4m3"]:
        x = (x * 4).to(torch.float8_e4m3fn)
    return x.transpose(1, 2) if case["head_major"] else x


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    i32 = dict(dtype=torch.int32, device=dev)
    s = {"case": dict(case)}
    if case["op"] == "map":
        old, new = _lengths(case)
        s["kv_len"], s["q_len"] = torch.tensor(old, **i32), torch.tensor(new, **i32)
        page = case["page"]
        need = [-(-(o + n) // page) - -(-o // page) for o, n in zip(old, new)]
        table, left, n_pages = _table(old, [0] * len(old), page, g, dev, sum(need) + 7)
        width = max(-(-(o + n) // page) for o, n in zip(old, new)) + 1
        wide = torch.full((case["B"], width), -1, **i32)
        w = min(width, table.shape[1])
        wide[:, :w] = table[:, :w]
        T = sum(new) + case["pad"]
        s |= {"table": wide, "free": left, "T": T, "kv_new": torch.empty(case["B"], **i32),
              "cu": torch.empty(case["B"] + 1, **i32), "position": torch.empty(T, **i32),
              "slot": torch.empty(T, **i32), "used": torch.empty(1, **i32)}
        return s
    D, Hq, Hk = case["dim"], case["heads"], case["kv_heads"]
    scales = torch.rand(2, Hk, generator=g, device=dev) * 0.2 + 0.15
    s["k_scale"], s["v_scale"] = (scales[0], scales[1]) if case["e4m3"] else (None, None)
    if case["op"] == "rope":
        T = case["T"]
        n_pages = -(-T // case["page"]) + 3
        s["k_cache"], s["v_cache"] = (_cache(case, n_pages, g, dev, False) for _ in range(2))
        # the projections' output in one buffer, as it comes from one matrix product
        qkv = torch.randn(T, (Hq + 2 * Hk) * D, generator=g, device=dev).to(torch.bfloat16)
        s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
        s["k"] = qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        s["v"] = qkv[:, (Hq + Hk) * D:].view(T, Hk, D)
        s["position"] = torch.randint(0, case["kv"], (T,), generator=g, **i32)
        s["slot"] = torch.randperm(n_pages * case["page"], generator=g, device=dev)[:T].to(torch.int32)
        s["q_norm"] = s["k_norm"] = None
        if case["norm"]:
            s["q_norm"] = torch.rand(D, generator=g, device=dev) + 0.5
            s["k_norm"] = torch.rand(D, generator=g, device=dev) + 0.5
        i = torch.arange(case["rot"] // 2, dtype=torch.float64, device=dev)
        s["inv_freq"] = torch.exp(-math.log(1e6) * 2 * i / case["rot"]).float()
        s["rot_scale"] = 1.0 if case["kv"] <= 32768 else 0.1 * math.log(case["kv"] / 32768) + 1.0
        s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
        return s
    old, new = _lengths(case)
    table, _, n_pages = _table(old, new, case["page"], g, dev, 2)
    T = sum(new)
    s["k_cache"], s["v_cache"] = (_cache(case, n_pages, g, dev, True) for _ in range(2))
    s["q"] = (torch.randn(T, Hq, D, generator=g, device=dev) * 1.5).to(torch.bfloat16)
    s["kv_len"] = torch.tensor([o + n for o, n in zip(old, new)], **i32)
    s["cu"] = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), **i32)
    s["table"] = table
    s["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=dev) / Hq) if case["slopes"] else None
    pre = case.get("prefix", 0)
    s["prefix"] = torch.full((case["B"],), pre, **i32) if pre else None
    s["scale"] = D ** -0.5
    s["most_q"], s["most_kv"] = max(new), max(o + n for o, n in zip(old, new))
    s["out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
    s["lse"] = torch.empty(T, Hq, dtype=torch.float32, device=dev)
    return s


# ---------------------------------------------------------------- the framework's calls

def _handle(s):
    """The cache descriptor and the workspace, which a user's program makes once and keeps beside its cache."""
    if "desc" not in s:
        import quantized_expert_ffn_top10_b200 as M
        c = s["case"]
        s["M"] = M
        s["desc"] = None
        if c["op"] != "map":
            s["desc"] = M.moe_kv_desc(s["k_cache"], s["v_cache"], c["heads"], s["k_scale"], s["v_scale"])
        if c["op"] in ("decode", "prefill"):
            n = M.moe_attn_workspace_bytes(s["q"].shape[0], c["B"], c["heads"], c["kv_heads"], c["dim"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s["M"], s["desc"]


def _own(s):
    M, desc = _handle(s)
    c = s["case"]
    if c["op"] == "map":
        M.moe_kv_map(s["kv_len"], s["q_len"], c["page"], s["free"], s["table"], s["kv_new"], s["cu"], s["position"],
                     s["slot"], s["used"])
        return _map_outputs(s)
    if c["op"] == "rope":
        M.moe_qk_norm_rope(desc, s["q"], s["k"], s["v"], s["position"], s["slot"], s["q_out"], s["inv_freq"],
                           q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6, rot_scale=s["rot_scale"],
                           interleaved=c["interleaved"])
        return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}
    if c["op"] == "decode":
        M.moe_attn_decode(desc, s["q"], s["cu"], s["kv_len"], s["table"], s["out"], c["q"], s["ws"], s["scale"],
                          softcap=c["softcap"], window=c["window"], slopes=s["slopes"], prefix=s["prefix"],
                          lse=s["lse"])
    else:
        M.moe_attn_prefill(desc, s["q"], s["cu"], s["kv_len"], s["table"], s["out"], s["ws"], s["scale"],
                           softcap=c["softcap"], window=c["window"], slopes=s["slopes"], prefix=s["prefix"],
                           lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- the plain forms

def _map_outputs(s):
    return {"table": s["table"], "kv_len": s["kv_new"], "cu": s["cu"], "position": s["position"], "slot": s["slot"],
            "used": s["used"]}


def _plain_map(s):
    page, old, new, free = s["case"]["page"], s["kv_len"].long(), s["q_len"].long(), s["free"]
    B, width = s["table"].shape
    have = (old + page - 1) // page
    want = (old + new + page - 1) // page
    room = want <= width
    need = torch.where(room, want - have, 0)
    upto = torch.cumsum(need, 0)
    granted = room & ((need == 0) | (upto <= free.numel()))
    col = torch.arange(width, device=old.device)[None]
    fresh = granted[:, None] & (col >= have[:, None]) & (col < want[:, None])
    at = ((upto - need - have)[:, None] + col).clamp(0, free.numel() - 1)
    s["table"].copy_(torch.where(fresh, free[at], s["table"]))
    s["cu"][0] = 0
    s["cu"][1:] = torch.cumsum(new, 0)
    t = torch.arange(s["T"], device=old.device)
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    live = b < B
    b = b.clamp(max=B - 1)
    pos = old[b] + t - s["cu"][b]
    slot = s["table"][b, (pos // page).clamp(max=width - 1)].long() * page + pos % page
    s["position"].copy_(torch.where(live, pos, 0))
    s["slot"].copy_(torch.where(live & granted[b], slot, -1))
    s["kv_new"].copy_(torch.where(granted, old + new, old))
    s["used"].copy_(torch.where(granted, need, 0).sum().reshape(1))
    return _map_outputs(s)


def _turned(x, cos, sin, interleaved):
    """x [T, heads, rot] turned by the angles of each token."""
    c, n = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat((a * c - b * n, b * c + a * n), -1)


def _rope_values(s, wide):
    """Normed and turned queries and keys, and the values, in `wide` floats."""
    c = s["case"]
    rot = c["rot"]
    angle = s["position"].double()[:, None] * s["inv_freq"].double()[None]
    cos, sin = ((f(angle) * s["rot_scale"]).to(wide) for f in (torch.cos, torch.sin))

    def one(x, w):
        x = x.to(wide)
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.to(wide)
        return torch.cat((_turned(x[..., :rot], cos, sin, c["interleaved"]), x[..., rot:]), -1)

    return one(s["q"], s["q_norm"]), one(s["k"], s["k_norm"]), s["v"].to(wide)


def _plain_rope(s):
    page = s["case"]["page"]
    q, k, v = _rope_values(s, torch.float32)
    s["q_out"].copy_(q)
    at = s["slot"].long()
    for cache, x, scale in ((s["k_cache"], k, s["k_scale"]), (s["v_cache"], v, s["v_scale"])):
        if scale is not None:
            x = (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
            cache.view(torch.uint8)[at // page, at % page] = x
        else:
            cache[at // page, at % page] = x.to(torch.bfloat16)
    return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}


def _gathered(cache, pages, offset, scale, live):
    """The cached rows of each request in order [B, S, heads, dim], in 32 bits; zero behind its length."""
    if scale is None:
        x = cache[pages, offset].float()
    else:
        x = cache.view(torch.uint8)[pages, offset].view(torch.float8_e4m3fn).float() * scale[:, None]
    return torch.where(live[..., None, None], x, 0.0)


def _plain_attention(s):
    c = s["case"]
    Hq, Hk, D, page = c["heads"], c["kv_heads"], c["dim"], c["page"]
    G = Hq // Hk
    S, Tm = s["most_kv"], s["most_q"]
    dev = s["q"].device
    kv, cu = s["kv_len"].long(), s["cu"].long()
    B = kv.numel()
    n = cu[1:] - cu[:-1]
    j = torch.arange(S, device=dev)
    live = j[None] < kv[:, None]
    pages = torch.where(live, s["table"][:, j // page], 0).long()
    offset = (j % page).expand(B, S)
    k = _gathered(s["k_cache"], pages, offset, s["k_scale"], live).permute(0, 2, 3, 1)  # [B, Hk, D, S]
    v = _gathered(s["v_cache"], pages, offset, s["v_scale"], live).permute(0, 2, 1, 3)  # [B, Hk, S, D]
    i = torch.arange(Tm, device=dev)
    row = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(B, Tm, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * Tm, D)
    x = (q @ k).view(B, Hk, G, Tm, S)
    x *= s["scale"]
    if c["softcap"]:
        x = torch.tanh(x / c["softcap"]) * c["softcap"]
    pos = (kv - n)[:, None] + i
    if s["slopes"] is not None:
        x = x - s["slopes"].view(1, Hk, G, 1, 1) * (pos[:, :, None] - j).abs()[:, None, None]
    last = pos + 1
    if s["prefix"] is not None:
        last = torch.maximum(last, torch.minimum(s["prefix"].long(), kv)[:, None])
    seen = (j < last[..., None]) & live[:, None]
    if c["window"]:
        seen &= j > pos[..., None] - c["window"]
    seen = seen[:, None, None]
    x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x = torch.exp_(x.sub_(top))
    total = x.sum(-1, keepdim=True)
    o = (x.view(B, Hk, G * Tm, S) @ v).view(B, Hk, G, Tm, D)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (torch.log(total) + top).squeeze(-1)
    t = torch.arange(s["q"].shape[0], device=dev)
    b = torch.searchsorted(cu[1:], t, right=True)
    t = t - cu[b]
    s["out"].copy_(o.permute(0, 3, 1, 2, 4)[b, t].view(s["out"].shape))
    s["lse"].copy_(lse.permute(0, 3, 1, 2)[b, t].view(s["lse"].shape))
    return {"out": s["out"], "lse": s["lse"]}


def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    return _plain_map(s) if op == "map" else _plain_rope(s) if op == "rope" else _plain_attention(s)


# ---------------------------------------------------------------- exact values

def _exact_rope(s):
    """The definition, a pair of elements at a time, in 64 bits."""
    c = s["case"]
    rot, page = c["rot"], c["page"]
    res = []
    for x, w in ((s["q"], s["q_norm"]), (s["k"], s["k_norm"])):
        y = x.double().clone()
        if w is not None:
            y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / c["dim"] + 1e-6) * w.double()
        z = y.clone()
        for p in range(rot // 2):
            a, b = (2 * p, 2 * p + 1) if c["interleaved"] else (p, p + rot // 2)
            angle = s["position"].double() * float(s["inv_freq"][p])
            turn = torch.polar(torch.full_like(angle, s["rot_scale"]), angle)[:, None]
            w2 = torch.complex(y[..., a], y[..., b]) * turn
            z[..., a], z[..., b] = w2.real, w2.imag
        res.append(z)
    out = {"q": res[0]}
    for name, x, scale in (("k", res[1], s["k_scale"]), ("v", s["v"].double(), s["v_scale"])):
        cache = s[name + "_cache"].double().clone()
        y = x if scale is None else (x / scale.double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        cache[s["slot"].long() // page, s["slot"].long() % page] = y
        out[name] = cache
    return out


def _exact_attention(s):
    """Request by request and cached head by cached head, in 64 bits."""
    c = s["case"]
    Hq, Hk, page = c["heads"], c["kv_heads"], c["page"]
    G = Hq // Hk
    q = s["q"].double()
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    cu = s["cu"].tolist()
    for b, rows in enumerate(_rows(c)):
        kv = int(s["kv_len"][b])
        where = torch.tensor([int(x) for x in s["table"][b, :-(-kv // page)].tolist()], device=q.device)
        first = torch.tensor([l for l, _ in rows], device=q.device)[:, None]
        last = torch.tensor([h for _, h in rows], device=q.device)[:, None]
        at = torch.arange(kv, device=q.device)[None]
        hidden = (at < first) | (at >= last)
        pos = torch.arange(kv - len(rows), kv, device=q.device)[:, None]
        for h in range(Hk):
            kv_rows = []
            for cache, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
                x = cache[:, :, h].view(torch.uint8)[where].view(cache.dtype).double().flatten(0, 1)[:kv]
                kv_rows.append(x if scale is None else x * scale[h].double())
            for g in range(G):
                head = h * G + g
                a = torch.mm(q[cu[b]:cu[b + 1], head], kv_rows[0].T) * s["scale"]
                if c["softcap"]:
                    a = c["softcap"] * torch.tanh(a / c["softcap"])
                if s["slopes"] is not None:
                    a -= s["slopes"][head].double() * (pos - at).abs()
                a[hidden] = -math.inf
                z = torch.logsumexp(a, -1)
                out[cu[b]:cu[b + 1], head] = torch.mm(torch.exp(a - z[:, None]), kv_rows[1])
                lse[cu[b]:cu[b + 1], head] = z
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "map":
        return None
    return _exact_rope(s) if case["op"] == "rope" else _exact_attention(s)
