"""One decoder attention block on the library's calls, as a program that verifies drafted tokens runs them:

    q, k, v = x Wqkv^T          qmv_q4_0 (up to eight tokens) or qmm_q4_0_prefill, Q4_0 weights
    pages, slots, positions     qmv_kv_pages
    rotate, write k and v       qmv_kv_append
    attention over the cache    qmv_tree_attn
    y = a Wo^T                  qmv_q4_0 / qmm_q4_0_prefill

A step takes any number of new tokens for each request: a prompt, one token, or a tree of drafted ones.  Every size on
the device side is fixed by the host's shapes, so a step with fixed shapes can be captured in a CUDA graph.

Behind the output head a tree of drafted tokens is verified without a host read:

    logits = h Whead^T          qmv_q4_0 or qmm_q4_0_prefill
    a token at each node        qmv_sample
    the path they accept        qmv_tree_accept
    its rows kept               qmv_kv_keep

    python -m weight_quantized_decode_gb300.decode_block        # prompt, tree, accepted path; checks and times them
"""
from __future__ import annotations

import numpy as np

import weight_quantized_decode_gb300 as qmv
from weight_quantized_decode_gb300 import synth


class AttentionBlock:
    """Q4_0 tables Wqkv [(heads + 2 kv_heads) * head_dim, hidden] and Wo [hidden, heads * head_dim] (uint8 CUDA tensors)
    and a paged cache for `requests` requests of at most `width` pages each; q_norm, k_norm: weights of the norms of query
    and key heads, where the model has them."""

    def __init__(self, Wqkv, Wo, hidden, heads, kv_heads, head_dim, requests, n_pages, width, page=32, q8=False,
                 base=10000.0, positions=8192, q_norm=None, k_norm=None, eps=1e-6):
        import torch
        self.torch = torch
        self.Wqkv, self.Wo, self.heads, self.page = Wqkv, Wo, heads, page
        self.cache = qmv.qmv_kv_cache(n_pages, kv_heads, page, head_dim, torch.int8 if q8 else torch.float16)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = torch.full((requests, width), -1, **i32)
        self.lens = torch.zeros(requests, **i32)
        self.free = torch.randperm(n_pages, device="cuda").to(torch.int32)
        self.head = torch.zeros(1, **i32)
        self.held = torch.zeros(requests, **i32)      # pages of each request, also past its length
        turn = base ** (-torch.arange(0, head_dim, 2, dtype=torch.float64, device="cuda") / head_dim)
        angle = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * turn
        self.cos, self.sin = angle.cos().float(), angle.sin().float()
        self.norms = dict(q_norm=q_norm, k_norm=k_norm, eps=eps)
        self.work = qmv.qmv_tree_attn_workspace()

    def _product(self, W, x):
        return qmv.qmv_q4_0(W, x) if x.shape[0] <= 8 else qmv.qmm_q4_0_prefill(W, x)

    def step(self, x, n_new, tree=None):
        """x fp16 [T, hidden]: the requests' new tokens, one request after another; n_new int32 [requests]; tree as
        qmv_tree_attn takes it.  Returns (y fp32 [T, hidden], maps).  The new tokens stay in the cache."""
        T = x.shape[0]
        qkv = self._product(self.Wqkv, x)
        maps = qmv.qmv_kv_pages(self.lens, n_new, self.free, self.table, self.page, T, head=self.head, tree=tree,
                                n_pages=self.cache.n_pages, held=self.held)
        q = qmv.qmv_kv_append(qkv, self.cache, maps.slots, self.heads, pos=maps.pos, cos=self.cos, sin=self.sin,
                              **self.norms)
        a = qmv.qmv_tree_attn(q, self.cache, self.table, maps.start, maps.kv_len, tree=tree, workspace=self.work)
        y = self._product(self.Wo, a.view(T, -1))
        self.lens, self.head, self.held = maps.kv_len, maps.head, maps.held
        return y, maps

    def keep(self, request, maps, path):
        """After a tree step: of `request`'s new tokens only the nodes of `path` (indices, root first) stay, in that
        order, and its length ends behind them.  The others' pages stay with the request (`held`), for its next tokens."""
        torch, page = self.torch, self.page
        start = int(maps.start[request])
        slots = maps.slots[start:int(maps.start[request + 1])].long()
        if bool((slots < 0).any()):
            raise RuntimeError("keep: the step had no pages for some of the request's tokens; nothing of it can be kept")
        frm, to = slots[torch.as_tensor(path, device="cuda")], slots[:len(path)]
        for pool in (self.cache.k, self.cache.v, self.cache.k_scale, self.cache.v_scale):
            if pool is not None:
                pool[to // page, :, to % page] = pool[frm // page, :, frm % page].clone()
        self.lens = self.lens.clone()
        self.lens[request] += len(path) - slots.numel()

    def accept(self, tokens, sampled, maps, tree=None):
        """After a tree step of all requests: the path that the tokens sampled at the nodes accept stays, for each of them,
        as `keep` does it, but without a host read.  Where the step had no pages for some of a request's nodes (a device
        status bit; `keep` refuses it) the path ends in front of them, and its length there; one whose first node had none
        keeps the length it had, with a count of 0.  Returns TreeAccepted; its `next` are the next step's first tokens, -1
        for a request without one: nothing new in the step, no page for its first node, or nothing that could be drawn at the
        last node of its path (logits that are -inf or no numbers, as where the attention met a missing page)."""
        got = qmv.qmv_tree_accept(tokens, sampled, maps.start, maps.kv_len, tree=tree, slots=maps.slots)
        qmv.qmv_kv_keep(self.cache, maps.slots, maps.start, got.path, got.count)
        self.lens = got.lens
        return got


class Decoder:
    """An embedding (fp16 [vocabulary, hidden]), an AttentionBlock and an output head (Q4_0 [vocabulary, hidden], no more
    tokens than the embedding): from token ids to the next ones on the GPU."""

    def __init__(self, block, embedding, head):
        if head.numel() > embedding.shape[0] * (embedding.shape[1] // 32 * qmv.Q4_0_BLOCK_BYTES):
            raise ValueError("Decoder: the head has more tokens than the embedding")
        self.block, self.embedding, self.head = block, embedding, head

    def logits(self, tokens, n_new, tree=None):
        """The requests' new tokens (int32 [T], as AttentionBlock.step takes them) through the model.  Returns (logits fp32
        [T, vocabulary], maps).  A token of -1, none, is looked up as token 0: `next` of an earlier step can be given as it
        is, but what a request without a token draws there means nothing (give it no new tokens, or finish it)."""
        x = self.embedding.index_select(0, tokens.clamp(min=0))
        y, maps = self.block.step(x, n_new, tree)
        return self.block._product(self.head, (x + y).half()), maps

    def step(self, tokens, n_new, u, tree=None, **settings):
        """`logits`, and a token drawn at each place by u [T] and qmv_sample's settings.  Returns (Sampled, maps)."""
        logits, maps = self.logits(tokens, n_new, tree)
        return qmv.qmv_sample(logits, u, **settings), maps

    def verify(self, tokens, n_new, u, tree=None, **settings):
        """A step of drafted trees, of which the accepted paths stay in the cache.  Returns TreeAccepted."""
        drawn, maps = self.step(tokens, n_new, u, tree, **settings)
        return self.block.accept(tokens, drawn.token, maps, tree)


def tree_mask(parents):
    """Mask words (int32 [nodes, ceil(nodes / 32)]) of a tree given by each node's parent (-1: the context)."""
    n = len(parents)
    seen = np.zeros((n, 32 * ((n + 31) // 32)), dtype=bool)
    for i, p in enumerate(parents):
        if p >= 0:
            seen[i] = seen[p]
        seen[i, i] = True
    return np.packbits(seen, axis=-1, bitorder="little").view(np.int32)


def main() -> int:
    import torch
    hidden, heads, kv_heads, D, prompt = 4096, 32, 8, 128, 1000
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    Wqkv = dev(synth.q4_0_weights((heads + 2 * kv_heads) * D, hidden, 1))
    Wo = dev(synth.q4_0_weights(hidden, heads * D, 2))
    parents = [-1, 0, 0, 1, 1, 2, 3, 6]
    path = [0, 1, 3, 6, 7]
    mask = dev(tree_mask(parents))
    one = lambda n: torch.tensor([n], dtype=torch.int32, device="cuda")  # noqa: E731
    for q8 in (False, True):
        g = torch.Generator(device="cuda").manual_seed(3)
        x = torch.randn(prompt + len(parents) + 1, hidden, generator=g, device="cuda").half()
        tree, chain = (AttentionBlock(Wqkv, Wo, hidden, heads, kv_heads, D, 1, 64, 64, q8=q8) for _ in range(2))
        for block in (tree, chain):
            block.step(x[:prompt], one(prompt))
        y, maps = tree.step(x[prompt:-1], one(len(parents)), tree=mask)
        tree.keep(0, maps, path)
        # the same path, one token at a time
        far = 0.0
        for node in path:
            y1, _ = chain.step(x[prompt + node:prompt + node + 1], one(1))
            far = max(far, float((y1 - y[node]).norm() / y1.norm()))
        # and the token after it, behind the kept path and behind the chain
        a, _ = tree.step(x[-1:], one(1))
        b, _ = chain.step(x[-1:], one(1))
        after = float((a - b).norm() / b.norm())
        bad = qmv.qmv_device_status()
        # a captured tree step
        block = tree
        state = block.lens, block.head, block.held
        side = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            block.step(x[prompt:-1], one(len(parents)), tree=mask)
            block.lens, block.head, block.held = state
            n_new = one(len(parents))
            side.synchronize()
            with torch.cuda.graph(graph, stream=side):
                block.step(x[prompt:-1], n_new, tree=mask)
            e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            for _ in range(3):
                graph.replay()
            e0.record(side)
            for _ in range(50):
                graph.replay()
            e1.record(side)
            side.synchronize()
        print(f"{'int8' if q8 else 'fp16'} cache: tree against chain {far:.1e}, next token {after:.1e}, status {bad}, "
              f"tree step of {len(parents)} nodes {e0.elapsed_time(e1) / 50 * 1e3:.1f} us")
        # (one token and eight run on different product kernels, whose fp16 partial sums differ)
        if bad or far > 1e-2 or after > 1e-2:
            return 1
    return drafted()


def agree(truth, rows, said, seen, limit=1e-2):
    """Whether two ways to the same tokens agree: truth[i] was drawn greedily from logits rows[i], said[i] from seen[i].  Rows
    may be `limit` apart, relative to their norm, and two tokens may change places whose logits differ by less than the
    rows do; behind such a pair the ways part, and no more is compared."""
    for t, a, s, b in zip(truth, rows, said, seen):
        if not float((a - b).norm()) <= limit * float(a.norm()):
            return False
        if t != s:
            return float(a[t] - a[s]) <= 2 * float((a - b).abs().max())
    return True


def drafted() -> int:
    """Drafted trees verified by their samples, against the same tokens decoded one by one (on other product kernels, so
    that two nearly equal logits may change places)."""
    import torch
    hidden, heads, kv_heads, D, vocab = 2048, 16, 8, 128, 32000
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(5)
    Wqkv, Wo = dev(synth.q4_0_weights((heads + 2 * kv_heads) * D, hidden, 4)), dev(synth.q4_0_weights(hidden, heads * D, 5))
    head = dev(synth.q4_0_weights(vocab, hidden, 6))
    embedding = torch.randn(vocab, hidden, generator=g, device="cuda").half()
    norms = [1 + 0.1 * torch.randn(D, generator=g, device="cuda") for _ in range(2)]
    one, two = (Decoder(AttentionBlock(Wqkv, Wo, hidden, heads, kv_heads, D, 1, 64, 64, q_norm=norms[0], k_norm=norms[1]),
                        embedding, head) for _ in range(2))
    count = lambda n: torch.tensor([n], dtype=torch.int32, device="cuda")  # noqa: E731
    prompt = torch.randint(0, vocab, (50,), generator=g, device="cuda", dtype=torch.int32)
    greedy = lambda logits: qmv.qmv_sample(logits, torch.zeros(len(logits), device="cuda"), temperature=0.0).token  # noqa: E731
    # eight tokens, one at a time
    logits, _ = one.logits(prompt, count(50))
    truth, rows = [int(greedy(logits)[-1])], [logits[-1]]
    for _ in range(8):
        logits, _ = one.logits(count(truth[-1]), count(1))
        truth.append(int(greedy(logits)[0]))
        rows.append(logits[0])
    # the same by trees in which the draft is right for three tokens and then wrong
    logits, _ = two.logits(prompt, count(50))
    said, seen, right = [int(greedy(logits)[-1])], [logits[-1]], True
    parents = [-1, 0, 0, 1, 1, 4, 5, 2]
    mask = dev(tree_mask(parents))
    while len(said) < 7:
        t = truth[len(said):] + [0] * 4
        nodes = [said[-1], t[0], 1, 2, t[1], t[2], (t[3] + 1) % vocab, 3]
        tokens = torch.tensor(nodes, dtype=torch.int32, device="cuda")
        logits, maps = two.logits(tokens, count(8), mask)          # (what Decoder.verify does, logits in hand)
        drawn = greedy(logits)
        got = two.block.accept(tokens, drawn, maps, mask)
        drew, path = drawn.tolist(), [0]
        while True:
            child = [j for j in range(8) if parents[j] == path[-1] and nodes[j] == drew[path[-1]]]
            if not child:
                break
            path.append(child[0])
        right = right and got.path.tolist() == path + [-1] * (8 - len(path)) and got.count.tolist() == [len(path)] and \
            got.next.tolist() == [drew[path[-1]]]
        said += [nodes[j] for j in path[1:]] + [drew[path[-1]]]
        seen += [logits[j] for j in path]
        print(f"tree of 8 nodes: {int(got.count[0])} accepted, next token {int(got.next[0])}")
    bad = qmv.qmv_device_status()
    same = agree(truth, rows, said, seen)
    print(f"one by one {truth[:len(said)]}, by trees {said[:len(truth)]}, {'agreed' if same else 'not the same'}, paths "
          f"{'as drawn' if right else 'wrong'}, status {bad}")
    return 0 if same and right and not bad else 1


if __name__ == "__main__":
    raise SystemExit(main())
