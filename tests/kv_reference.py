"""Plain 64-bit forms of the paged-cache calls (numpy), and the problems the
GPU tests give them.  None of this is used by the product path."""
import numpy as np


def pages(lens, news, free, table, page, tokens, head=0, tree=None):
    """Page and slot maps, one request after another: a dict of arrays."""
    table = table.copy()
    start, kv_len, slots, pos, req = [0], [], [], [], []
    at = head
    for r, (a, n) in enumerate(zip(lens, news)):
        n = min(int(n), tokens - start[-1])
        have, need = -(-int(a) // page), -(-(int(a) + n) // page)
        for j in range(have, need):
            if j < table.shape[1]:
                table[r, j] = free[at] if at < len(free) else -1
            at += 1
        for i in range(n):
            w = int(a) + i
            p = table[r, w // page] if w // page < table.shape[1] else -1
            slots.append(p * page + w % page if p >= 0 else -1)
            if tree is None:
                pos.append(w)
            else:
                row = tree[start[-1] + i]
                bits = [j for j in range(min(n, 32 * len(row))) if int(row[j // 32]) >> (j % 32) & 1]
                pos.append(int(a) + max(0, len(bits) - 1))
            req.append(r)
        start.append(start[-1] + n)
        kv_len.append(int(a) + n)
    pad = tokens - len(slots)
    return {"table": table, "start": start, "kv_len": kv_len, "slots": slots + [-1] * pad, "pos": pos + [0] * pad,
            "request": req + [-1] * pad, "head": [min(at, len(free))]}


def rotate(x, rot, interleaved, cos, sin):
    """x [..., D] float64; cos, sin [..., rot / 2] broadcastable."""
    y = np.array(x)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        y[..., a] = x[..., a] * cos[..., i] - x[..., b] * sin[..., i]
        y[..., b] = x[..., b] * cos[..., i] + x[..., a] * sin[..., i]
    return y


def random_trees(news, words, rs):
    """int32 [sum(news), words]: each node sees itself and its ancestors."""
    rows = []
    for n in news:
        seen = np.zeros((n, 32 * words), dtype=bool)
        for i in range(n):
            parent = rs.randint(max(-1, i - 6), i) if i else -1
            if parent >= 0:
                seen[i] = seen[parent]
            seen[i, i] = True
        rows.append(seen)
    seen = np.concatenate(rows) if rows else np.zeros((0, 32 * words), dtype=bool)
    return np.packbits(seen, axis=-1, bitorder="little").view(np.int32).reshape(-1, words)


def sees(node, nodes, length, tree_row):
    """Which of `length` places a request's node sees (bool array)."""
    ctx = length - nodes
    s = np.ones(length, dtype=bool)
    for j in range(nodes):
        if tree_row is None:
            s[ctx + j] = j <= node
        else:
            s[ctx + j] = j < 32 * len(tree_row) and bool(int(tree_row[j // 32]) >> (j % 32) & 1)
    return s


def attention(prob, scale):
    """(out, allowance), float64 [T, Hq, D].

    The allowance follows from the arithmetic.  The output is rounded to fp16
    (2^-11 |o|, or half a subnormal step 2^-25).  Each weight p = exp(s - max)
    is rounded to fp16 (2^-11 of it; or, kept above 2^-14 only after a scaling
    by 2^10 against the largest row scale, an absolute 2^-35 of it), and carries
    the fp32 error of its score: the sum of D products, each rounding at most
    2^-24 of the sum of magnitudes, and a few roundings of the scaled score and
    of exp2.  With A = sum p |v| / sum p the output moves by at most
    (2^-11 + 2 E) A; the factor 2 covers the sum in the denominator."""
    out = np.zeros((prob["q"].shape[0],) + prob["q"].shape[1:], dtype=np.float64)
    allow = np.zeros_like(out)
    start, heads, hk = prob["start"], prob["q"].shape[1], prob["k"].shape[1]
    D, page, group = prob["q"].shape[2], prob["k"].shape[2], heads // hk
    for r in range(len(prob["kv_len"])):
        nodes, length = int(start[r + 1] - start[r]), int(prob["kv_len"][r])
        if nodes == 0:
            continue
        ids = prob["table"][r, :-(-length // page)]
        k = prob["k"][ids].astype(np.float64)
        v = prob["v"][ids].astype(np.float64)
        if prob["k_scale"] is not None:
            k = k * prob["k_scale"][ids].astype(np.float64)[..., None]
            v = v * prob["v_scale"][ids].astype(np.float64)[..., None]
        k = k.transpose(1, 0, 2, 3).reshape(hk, -1, D)[:, :length]
        v = v.transpose(1, 0, 2, 3).reshape(hk, -1, D)[:, :length]
        for i in range(nodes):
            t = int(start[r]) + i
            s = sees(i, nodes, length, None if prob["tree"] is None else prob["tree"][t])
            if not s.any():
                continue
            for h in range(heads):
                kk, vv = k[h // group][s], v[h // group][s]
                q = prob["q"][t, h].astype(np.float64)
                score = kk @ q * scale
                p = np.exp(score - score.max())
                total = p.sum()
                out[t, h] = p @ vv / total
                sums = (np.abs(kk) @ np.abs(q)).max() * abs(scale)
                E = (D + 8) * 2.0 ** -24 * sums + 2.0 ** -20
                A = p @ np.abs(vv) / total
                allow[t, h] = 2.0 ** -11 * np.abs(out[t, h]) + (2.0 ** -11 + 2 * E) * A \
                    + 2.0 ** -25 + len(p) * 2.0 ** -34 * np.abs(vv).max()
    return out, allow


def problem(lens, news, heads, hk, D, page, q8=False, tree=None, words=None, seed=0, width=None, spare=2, spread=1.0):
    """A cache with random pages, queries and maps.  tree: None (chain), "random", or an int32 array."""
    rs = np.random.RandomState(seed)
    total = [a + b for a, b in zip(lens, news)]
    used = [-(-t // page) for t in total]
    n_pages = sum(used) + spare
    perm = rs.permutation(n_pages)
    width = max(used + [1]) if width is None else width
    table = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for r, u in enumerate(used):
        table[r, :u] = perm[at:at + u]
        at += u
    T = sum(news)
    prob = {"q": rs.randn(T, heads, D).astype(np.float16), "table": table, "kv_len": np.array(total, dtype=np.int32),
            "start": np.concatenate([[0], np.cumsum(news)]).astype(np.int32), "k_scale": None, "v_scale": None}
    for name in ("k", "v"):
        x = (rs.randn(n_pages, hk, page, D) * (spread if name == "k" else 1.0)).astype(np.float32)
        if q8:
            d = (np.abs(x).max(-1) / 127).astype(np.float32)
            prob[name], prob[name + "_scale"] = np.rint(x / d[..., None]).astype(np.int8), d
        else:
            prob[name] = x.astype(np.float16)
    if isinstance(tree, str):
        words = max(1, -(-max(news + [1]) // 32)) if words is None else words
        tree = random_trees(news, words, rs)
    prob["tree"] = tree
    return prob
