"""Timed cases of the paged-cache operators: page and slot maps from request lengths, the rotary cache write, and
attention of drafted tokens over the cache.

Each operator has a plain form of elementary torch operations in 32 bits and the framework's call; `own` chooses.
Head layouts are those of the decoders whose weight tables the benchmark sweeps (hidden 4096: 32 query heads on 8
key/value heads of 128; 16 on 8 of 128) and a generic wide group (64 on 8 of 64).  A request has `len` tokens in the
cache and brings `new` ones: one token (plain decode), a tree of drafted tokens, or a chunk of a prompt.
"""
import math

import numpy as np
import torch

own = False

GOLD = 0.6180339887498949


# -- cases -------------------------------------------------------------------------


def listed():
    return [
        # Page and slot maps.  One stream that verifies a small tree: nothing but latency.
        {"name": "pages_one_tree", "op": "pages", "requests": 1, "len_lo": 1000, "len_hi": 1000, "new_lo": 8,
         "new_hi": 8, "page": 16, "tree": True},
        # A server admits many prompts of odd lengths at once: every new token gets its slot.
        {"name": "pages_prompts", "op": "pages", "requests": 1000, "len_lo": 0, "len_hi": 2000, "new_lo": 1,
         "new_hi": 509, "page": 64, "tree": False},
        # Cache write.  One token of a stacked query/key/value product in fp32, as the decode calls return it.
        {"name": "append_one", "op": "append", "tokens": 1, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "input": "f32", "cache": "f16", "page": 16, "interleaved": False},
        # The tokens of a batch of trees into an 8-bit cache, pairs rotated as neighbours.
        {"name": "append_trees_q8", "op": "append", "tokens": 517, "heads": 16, "kv_heads": 8, "dim": 128, "rot": 128,
         "input": "f16", "cache": "q8", "page": 32, "interleaved": True},
        # A long prompt at once: bandwidth.
        {"name": "append_prompt", "op": "append", "tokens": 16381, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "input": "f32", "cache": "f16", "page": 64, "interleaved": False},
        # Attention.  One token of one stream, moderate context: latency.
        {"name": "attend_one", "op": "attend", "requests": 1, "len_lo": 4095, "len_hi": 4095, "new_lo": 1, "new_hi": 1,
         "heads": 32, "kv_heads": 8, "dim": 128, "cache": "f16", "page": 16, "tree": False},
        # A small tree of one stream over a long, odd context.
        {"name": "attend_tree", "op": "attend", "requests": 1, "len_lo": 30001, "len_hi": 30001, "new_lo": 8,
         "new_hi": 8, "heads": 32, "kv_heads": 8, "dim": 128, "cache": "f16", "page": 32, "tree": True},
        # One token for each of many requests of uneven lengths, 8-bit cache.
        {"name": "attend_batch_q8", "op": "attend", "requests": 64, "len_lo": 100, "len_hi": 16383, "new_lo": 1,
         "new_hi": 1, "heads": 32, "kv_heads": 8, "dim": 128, "cache": "q8", "page": 32, "tree": False},
        # A batch of trees of uneven sizes, two query heads to a key/value head.
        {"name": "attend_batch_trees", "op": "attend", "requests": 16, "len_lo": 511, "len_hi": 8191, "new_lo": 1,
         "new_hi": 24, "heads": 16, "kv_heads": 8, "dim": 128, "cache": "f16", "page": 16, "tree": True},
        # Wide trees with a wide group: hundreds of rows share each key, arithmetic bounds it.
        {"name": "attend_wide_trees", "op": "attend", "requests": 8, "len_lo": 4001, "len_hi": 8001, "new_lo": 64,
         "new_hi": 64, "heads": 64, "kv_heads": 8, "dim": 64, "cache": "f16", "page": 64, "tree": True},
        # A tree over a very long context: one read of a gigabyte of keys and values.
        {"name": "attend_long", "op": "attend", "requests": 1, "len_lo": 262147, "len_hi": 262147, "new_lo": 16,
         "new_hi": 16, "heads": 32, "kv_heads": 8, "dim": 128, "cache": "f16", "page": 128, "tree": True},
        # Chunks of two prompts behind what is already cached, causal.
        {"name": "attend_chunks", "op": "attend", "requests": 2, "len_lo": 2000, "len_hi": 2800, "new_lo": 1400,
         "new_hi": 1500, "heads": 32, "kv_heads": 8, "dim": 128, "cache": "f16", "page": 64, "tree": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "append", "attend", "attend", "attend"])
    page = rng.choice([16, 32, 64, 128])
    if op == "pages":
        tree = rng.random() < 0.5
        requests = _log(rng, 1, 1000)
        hi = _log(rng, 1, 96 if tree else 509)
        return {"op": op, "requests": requests, "len_lo": rng.randint(0, 40), "len_hi": _log(rng, 41, 2000),
                "new_lo": rng.randint(1, hi), "new_hi": hi, "page": page, "tree": tree}
    heads, kv_heads, dim = rng.choice([(32, 8, 128), (16, 8, 128), (64, 8, 64), (12, 4, 64), (28, 4, 128), (8, 8, 128),
                                       (20, 1, 64)])
    cache = rng.choice(["f16", "q8"])
    if op == "append":
        return {"op": op, "tokens": _log(rng, 1, 16000), "heads": min(heads, 32), "kv_heads": kv_heads, "dim": dim,
                "rot": rng.choice([0, dim // 2, dim]), "input": rng.choice(["f32", "f16"]), "cache": cache,
                "page": page, "interleaved": rng.random() < 0.5}
    new = _log(rng, 1, 1500)
    if rng.random() < 0.4:
        new = rng.randint(1, 8)
    requests = _log(rng, 1, 64)
    # no more than the largest listed cases: tokens in the cache, and products
    per_token = 4.0 * heads * dim
    while requests > 1 and requests * new * new * per_token > 4e10:
        requests -= 1
    most = min(260000.0 * 1024 / (kv_heads * dim), 1.2e11 / (per_token * new)) / requests - new
    hi = _log(rng, 16, max(17.0, min(most, 200000.0)))
    return {"op": op, "requests": requests, "len_lo": rng.randint(0, hi) if requests > 1 else hi, "len_hi": hi,
            "new_lo": rng.randint(1, new) if requests > 1 else new, "new_hi": new, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "cache": cache, "page": page,
            "tree": new <= 128 and rng.random() < 0.6}


def _spread(lo, hi, n, phase):
    """n whole numbers between lo and hi, uneven, the same for every seed; one number alone is hi."""
    if n == 1:
        return [hi]
    return [lo + int((hi - lo + 1) * ((GOLD * (i + phase)) % 1.0)) for i in range(n)]


def _lens(case):
    return _spread(case["len_lo"], case["len_hi"], case["requests"], 1)


def _news(case):
    return _spread(case["new_lo"], case["new_hi"], case["requests"], 7)


# -- inputs ------------------------------------------------------------------------


def _rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2 + 1)
    return g


def _trees(news, seed):
    """Ancestor masks of random trees: bit j of a token's row is set where node j is its ancestor or itself.
    int32 words [tokens, ceil(most / 32)]."""
    most = max(news)
    words = (most + 31) // 32
    rs = np.random.RandomState(int(seed) % (1 << 31))
    n = len(news)
    seen = np.zeros((n, most, words * 32), dtype=bool)
    rows = np.arange(n)
    for i in range(most):
        parent = rs.randint(max(-1, i - 9), i, size=n) if i else np.full(n, -1)
        seen[:, i] = np.where((parent >= 0)[:, None], seen[rows, np.maximum(parent, 0)], False)
        seen[:, i, i] = True
    packed = np.packbits(seen, axis=-1, bitorder="little").view(np.int32)
    return np.concatenate([packed[r, :news[r]] for r in range(n)])


def _rows(shape, g, kind):
    """Rows as keys and values have them: unit spread, a few channels larger than the rest."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16)
    if kind == "k":
        x[..., :: max(1, shape[-1] // 4)] *= 3
    return x


def _quantised(x):
    """8-bit rows: codes and one fp32 scale to a row."""
    f = x.float()
    d = f.abs().amax(-1) / 127
    return torch.round(f / d.clamp_min(1e-30)[..., None]).to(torch.int8), d


def _inputs(case, seed):
    g = _rng(seed)
    s = {"case": case}
    if case["op"] == "pages":
        lens, news, page = _lens(case), _news(case), case["page"]
        width = max((a + b + page - 1) // page for a, b in zip(lens, news))
        n_pages = sum((a + b + page - 1) // page for a, b in zip(lens, news)) + 32
        perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        have = [(a + page - 1) // page for a in lens]
        table = np.full((len(lens), width), -1, dtype=np.int32)
        at, host = 0, perm.cpu().numpy()
        for r, h in enumerate(have):
            table[r, :h] = host[at:at + h]
            at += h
        s |= {"lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
              "news": torch.tensor(news, dtype=torch.int32, device="cuda"),
              "table": torch.from_numpy(table).cuda(), "free": perm[at:].contiguous(), "tokens": sum(news),
              "head": torch.full((1,), int(seed) % 5, dtype=torch.int32, device="cuda"),
              "tree": torch.from_numpy(_trees(news, seed)).cuda() if case["tree"] else None}
        return s
    hk, d, page, q8 = case["kv_heads"], case["dim"], case["page"], case["cache"] == "q8"
    if case["op"] == "append":
        n = case["tokens"]
        n_pages = n // page + 3
        kind = torch.float32 if case["input"] == "f32" else torch.float16
        s["qkv"] = torch.randn((n, (case["heads"] + 2 * hk) * d), generator=g, device="cuda", dtype=kind)
        s["slots"] = torch.randperm(n_pages * page, generator=g, device="cuda")[:n].to(torch.int32)
        s["pos"] = torch.randint(0, 8192, (n,), generator=g, device="cuda", dtype=torch.int32)
        s["cos"] = s["sin"] = None
        if case["rot"]:
            # the rotation tables of a program: one row to a position, computed once
            f = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
            a = torch.arange(8192, dtype=torch.float64, device="cuda")[:, None] * f
            s["cos"], s["sin"] = a.cos().float(), a.sin().float()
        for name in ("k", "v"):
            x = _rows((n_pages, hk, page, d), g, name)
            s[name], s[name + "_scale"] = _quantised(x) if q8 else (x, None)
        return s
    lens, news = _lens(case), _news(case)
    total = [a + b for a, b in zip(lens, news)]
    used = [(t + page - 1) // page for t in total]
    n_pages = sum(used) + 3
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    host = perm.cpu().numpy()
    table = np.full((len(lens), max(used)), -1, dtype=np.int32)
    stale, at = [], 0
    for r, u in enumerate(used):
        table[r, :u] = host[at:at + u]
        at += u
        stale += [int(table[r, u - 1]) * page + i for i in range((total[r] - 1) % page + 1, page)]
    for name in ("k", "v"):
        x = _rows((n_pages, hk, page, d), g, name)
        s[name], s[name + "_scale"] = _quantised(x) if q8 else (x, None)
        if stale:  # slots past a request's end hold whatever the memory held
            at_page = torch.tensor([t // page for t in stale], device="cuda")
            at_row = torch.tensor([t % page for t in stale], device="cuda")
            (s[name + "_scale"] if q8 else s[name])[at_page, :, at_row] = math.nan
    n = sum(news)
    start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    s |= {"q": torch.randn((n, case["heads"], d), generator=g, device="cuda", dtype=torch.float16),
          "table": torch.from_numpy(table).cuda(), "start": torch.from_numpy(start).cuda(),
          "kv_len": torch.tensor(total, dtype=torch.int32, device="cuda"), "most_new": max(news),
          "tree": torch.from_numpy(_trees(news, seed)).cuda() if case["tree"] else None, "work": None}
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import weight_quantized_decode_gb300 as fw
        if case["op"] != "pages":
            s["cache"] = fw.KvCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if case["op"] == "attend":
            s["work"] = fw.qmv_tree_attn_workspace()  # kept by a program from call to call
    return s


# -- one pass ----------------------------------------------------------------------


def run(s):
    return {"pages": _pages, "append": _append, "attend": _attend}[s["case"]["op"]](s)


def _stored(x, scale):
    """A cache as the values it stands for."""
    return x if scale is None else x.float() * scale[..., None]


def _pages(s):
    page = s["case"]["page"]
    if own:
        import weight_quantized_decode_gb300 as fw
        p = fw.qmv_kv_pages(s["lens"], s["news"], s["free"], s["table"], page, s["tokens"], head=s["head"],
                            tree=s["tree"])
        return {"table": s["table"], "start": p.start, "kv_len": p.kv_len, "slots": p.slots, "pos": p.pos,
                "request": p.request, "head": p.head}
    lens, news, table, n = s["lens"], s["news"], s["table"], s["tokens"]
    start = torch.cat([torch.zeros_like(news[:1]), news.cumsum(0, dtype=torch.int32)])
    kv_len = lens + news
    have, need = (lens + page - 1) // page, (kv_len + page - 1) // page
    more = need - have
    base = more.cumsum(0, dtype=torch.int32) - more + s["head"]
    j = torch.arange(table.shape[1], device="cuda", dtype=torch.int32)
    fresh = (j >= have[:, None]) & (j < need[:, None])
    at = (base[:, None] + j - have[:, None]).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(fresh, s["free"][at], table))
    t = torch.arange(n, device="cuda", dtype=torch.int32)
    request = torch.searchsorted(start, t, right=True, out_int32=True) - 1
    i = t - start[request]
    cached = lens[request]
    where = cached + i
    slots = table[request, where // page] * page + where % page
    pos = where
    if s["tree"] is not None:
        bits = (s["tree"][:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        pos = cached + bits.sum((1, 2), dtype=torch.int32) - 1
    return {"table": table, "start": start, "kv_len": kv_len, "slots": slots, "pos": pos, "request": request,
            "head": s["head"] + more.sum(dtype=torch.int32)}


def _turned(x, rot, interleaved, cos, sin):
    """Rotates the first `rot` values of each row: pairs (2i, 2i + 1) where interleaved, (i, i + rot / 2) where not."""
    if not rot:
        return x
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    c, d = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([c, d], -1).flatten(-2) if interleaved else torch.cat([c, d], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _append(s):
    case = s["case"]
    heads, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    if own:
        import weight_quantized_decode_gb300 as fw
        q = fw.qmv_kv_append(s["qkv"], s["cache"], s["slots"], heads, pos=s["pos"], cos=s["cos"], sin=s["sin"],
                             interleaved=case["interleaved"])
        return {"q": q, "k": _stored(s["k"], s["k_scale"]), "v": _stored(s["v"], s["v_scale"])}
    x = s["qkv"].float().view(-1, heads + 2 * hk, d)
    at = s["pos"].long()
    cos, sin = (s["cos"][at][:, None], s["sin"][at][:, None]) if case["rot"] else (None, None)
    q = _turned(x[:, :heads], case["rot"], case["interleaved"], cos, sin).half()
    k = _turned(x[:, heads:heads + hk], case["rot"], case["interleaved"], cos, sin)
    v = x[:, heads + hk:]
    slots = s["slots"].long()
    to, row = slots // page, slots % page
    _store(s["k"], s["k_scale"], to, row, k)
    _store(s["v"], s["v_scale"], to, row, v)
    return {"q": q, "k": _stored(s["k"], s["k_scale"]), "v": _stored(s["v"], s["v_scale"])}


def _store(pool, scale, to, row, x):
    if scale is None:
        pool[to, :, row] = x.half()
        return
    d = x.abs().amax(-1) / torch.full((1,), 127.0, device="cuda")
    y = x * torch.where(d > 0, torch.ones_like(d) / d, torch.zeros_like(d))[..., None]
    code = torch.trunc(y + torch.copysign(torch.full_like(y, 0.5), y))  # nearest, ties away from zero
    pool[to, :, row] = code.to(torch.int8)
    scale[to, :, row] = d


def _attend(s):
    case = s["case"]
    if own:
        import weight_quantized_decode_gb300 as fw
        return fw.qmv_tree_attn(s["q"], s["cache"], s["table"], s["start"], s["kv_len"], tree=s["tree"],
                                workspace=s["work"])
    heads, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    group, n, most = heads // hk, s["q"].shape[0], s["most_new"]
    start, kv_len = s["start"].long(), s["kv_len"].long()
    news = start[1:] - start[:-1]
    # every request's queries [R, T] and cached rows [R, L], padded
    node = torch.arange(most, device="cuda")
    token = (start[:-1, None] + node).clamp(max=n - 1)
    q = s["q"][token].float().view(-1, most, hk, group, d).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [R, hk, G T, D]
    pages = s["table"].clamp(min=0).long()
    k = _stored(s["k"][pages], s["k_scale"][pages] if s["k_scale"] is not None else None).float()
    v = _stored(s["v"][pages], s["v_scale"][pages] if s["v_scale"] is not None else None).float()
    k, v = k.transpose(1, 2).flatten(2, 3), v.transpose(1, 2).flatten(2, 3)  # [R, hk, L, D]
    at = torch.arange(k.shape[2], device="cuda")
    v = torch.where((at < kv_len[:, None])[:, None, :, None], v, torch.zeros((), device="cuda"))
    # which row sees which place: everything cached before the new tokens, and of those the ancestors
    there = at - (kv_len - news)[:, None]  # [R, L], the node at a place
    if s["tree"] is not None:
        words = s["tree"][token].long()  # [R, T, words]
        to = there.clamp(0, words.shape[2] * 32 - 1)
        bits = (words.gather(2, (to // 32)[:, None, :].expand(-1, most, -1)) >> (to % 32)[:, None, :]) & 1
        sees = (there < 0)[:, None, :] | ((bits != 0) & (at < kv_len[:, None])[:, None, :])
    else:
        sees = there[:, None, :] <= node[:, None]
    sees = sees & (at < kv_len[:, None])[:, None, :]
    score = (q @ k.transpose(2, 3)) * d ** -0.5
    score = score.view(-1, hk, group, most, at.numel())
    score = torch.where(sees[:, None, None], score, torch.full((), -math.inf, device="cuda"))
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(score - top)
    total = p.sum(-1)
    out = p.flatten(2, 3) @ v
    out = out.view(-1, hk, group, most, d) / torch.where(total > 0, total, torch.ones_like(total))[..., None]
    request = torch.searchsorted(s["start"], torch.arange(n, device="cuda", dtype=torch.int32), right=True) - 1
    out = out.permute(0, 3, 1, 2, 4)[request, torch.arange(n, device="cuda") - start[request]]
    return out.reshape(n, heads, d).half()


# -- what a pass cannot do without -------------------------------------------------


def work(case):
    if case["op"] == "pages":
        lens, news, page = _lens(case), _news(case), case["page"]
        more = sum((a + b + page - 1) // page - (a + page - 1) // page for a, b in zip(lens, news))
        words = (max(news) + 31) // 32 if case["tree"] else 0
        n = sum(news)
        # lengths and counts in, fresh pages from the list to the table, three numbers to a token
        return {"bytes": 4.0 * (2 * len(lens) + 2 * more + 2 * len(lens) + n * (3 + words)), "flops": 0.0}
    hk, d = case["kv_heads"], case["dim"]
    row = d + 4 if case["cache"] == "q8" else 2 * d
    if case["op"] == "append":
        n, heads = case["tokens"], case["heads"]
        wide = 4 if case["input"] == "f32" else 2
        return {"bytes": n * (float((heads + 2 * hk) * d * wide) + heads * d * 2 + 2 * hk * row + 8 + 4 * case["rot"]),
                "flops": 3.0 * n * (heads + hk) * case["rot"]}
    lens, news = _lens(case), _news(case)
    heads, n = case["heads"], sum(news)
    words = (max(news) + 31) // 32 if case["tree"] else 0
    pages = sum((a + b + case["page"] - 1) // case["page"] for a, b in zip(lens, news))
    moved = sum(a + b for a, b in zip(lens, news)) * 2.0 * hk * row + n * (4.0 * heads * d + 4 * words) + 4.0 * pages
    # a token sees what was cached and, at the least it can in a chain, the half of the new ones before it
    seen = sum(b * a + (b * (b + 1) / 2 if not case["tree"] else b) for a, b in zip(lens, news))
    return {"bytes": moved, "flops": 4.0 * heads * d * seen}


# -- the definition in 64 bits -----------------------------------------------------


def exact(case, seed):
    if case["op"] == "pages":
        return None  # whole numbers: compared as they are
    s = _inputs(case, seed)
    return (_exact_append if case["op"] == "append" else _exact_attend)(case, s)


def _exact_append(case, s):
    heads, hk, d, page, rot = case["heads"], case["kv_heads"], case["dim"], case["page"], case["rot"]
    x = s["qkv"].double().view(-1, heads + 2 * hk, d)
    if rot:
        turn = torch.complex(s["cos"].double(), s["sin"].double())[s["pos"].long()][:, None]
        part = x[:, :heads + hk, :rot]
        part = part.unflatten(-1, (rot // 2, 2)) if case["interleaved"] else part.unflatten(-1, (2, rot // 2)).mT
        z = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn)
        x = x.clone()
        x[:, :heads + hk, :rot] = (z if case["interleaved"] else z.mT).flatten(-2)
    out = {"q": x[:, :heads].contiguous()}
    slots = s["slots"].long()
    for name, first in (("k", heads), ("v", heads + hk)):
        rows = x[:, first:first + hk]
        pool = s[name].double()
        if s[name + "_scale"] is not None:
            pool = pool * s[name + "_scale"].double()[..., None]
            unit = rows.abs().amax(-1, keepdim=True) / 127
            rows = torch.where(unit > 0, (rows / unit.clamp_min(1e-300)).abs().add(0.5).floor() * rows.sign(), 0) * unit
        flat = pool.transpose(1, 2).reshape(-1, hk, d)
        flat[slots] = rows
        out[name] = flat.view(-1, page, hk, d).transpose(1, 2).contiguous()
    return out


def _exact_attend(case, s):
    heads, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    group = heads // hk
    lens, news = _lens(case), _news(case)
    out = torch.zeros((sum(news), heads, d), dtype=torch.float64, device="cuda")
    first = 0
    for r, (cached, new) in enumerate(zip(lens, news)):
        length = cached + new
        pages = s["table"][r, :(length + page - 1) // page].long()
        seen = torch.ones((new, length), dtype=torch.bool, device="cuda")
        if s["tree"] is None:
            seen[:, cached:] = torch.ones((new, new), dtype=torch.bool, device="cuda").tril()
        else:
            raw = s["tree"][first:first + new].cpu().numpy().view(np.uint8)
            bits = np.unpackbits(raw, axis=-1, bitorder="little")[:, :new].astype(bool)
            seen[:, cached:] = torch.from_numpy(bits).cuda()
        for h in range(hk):
            rows = {}
            for name in ("k", "v"):
                x = s[name][pages, h].reshape(-1, d)[:length].double()
                if s[name + "_scale"] is not None:
                    x = x * s[name + "_scale"][pages, h].reshape(-1)[:length, None].double()
                rows[name] = x
            for g in range(h * group, (h + 1) * group):
                score = s["q"][first:first + new, g].double() @ rows["k"].T / math.sqrt(d)
                out[first:first + new, g] = score.masked_fill(~seen, -math.inf).softmax(-1) @ rows["v"]
        first += new
    return out
