"""One decoder attention block on the library's calls, as a program that verifies drafted tokens runs them:

    q, k, v = x Wqkv^T          qmv_q4_0 (up to eight tokens) or qmm_q4_0_prefill, Q4_0 weights
    pages, slots, positions     qmv_kv_pages
    rotate, write k and v       qmv_kv_append
    attention over the cache    qmv_tree_attn
    y = a Wo^T                  qmv_q4_0 / qmm_q4_0_prefill

A step takes any number of new tokens for each request: a prompt, one token, or a tree of drafted ones.  Every size on
the device side is fixed by the host's shapes, so a step with fixed shapes can be captured in a CUDA graph.

    python -m weight_quantized_decode_gb300.decode_block        # prompt, tree, accepted path; checks and times them
"""
from __future__ import annotations

import numpy as np

import weight_quantized_decode_gb300 as qmv
from weight_quantized_decode_gb300 import synth


class AttentionBlock:
    """Q4_0 tables Wqkv [(heads + 2 kv_heads) * head_dim, hidden] and Wo [hidden, heads * head_dim] (uint8 CUDA tensors)
    and a paged cache for `requests` requests of at most `width` pages each."""

    def __init__(self, Wqkv, Wo, hidden, heads, kv_heads, head_dim, requests, n_pages, width, page=32, q8=False,
                 base=10000.0, positions=8192):
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
        q = qmv.qmv_kv_append(qkv, self.cache, maps.slots, self.heads, pos=maps.pos, cos=self.cos, sin=self.sin)
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
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
