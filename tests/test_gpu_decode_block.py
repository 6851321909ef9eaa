"""The attention block runs its calls together: a tree step gives what the
same tokens give one at a time, and goes on from an accepted path."""
import numpy as np
import pytest

from weight_quantized_decode_gb300 import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import weight_quantized_decode_gb300 as m
    m.lib()
    m.qmv_device_status()
    return m


def test_tree_mask():
    from weight_quantized_decode_gb300.decode_block import tree_mask
    m = tree_mask([-1, 0, 0, 2])
    assert m.shape == (4, 1) and m[:, 0].tolist() == [0b1, 0b11, 0b101, 0b1101]
    assert tree_mask([-1] * 33).shape == (33, 2)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("prompts", [[37], [100, 3, 64]])
def test_tree_step_equals_chains(q, q8, prompts):
    from weight_quantized_decode_gb300.decode_block import AttentionBlock, tree_mask
    hidden, heads, kv_heads, D = 512, 8, 2, 64
    Wqkv = torch.from_numpy(synth.q4_0_weights((heads + 2 * kv_heads) * D, hidden, 1)).cuda()
    Wo = torch.from_numpy(synth.q4_0_weights(hidden, heads * D, 2)).cuda()
    R = len(prompts)
    new = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    parents, path = [-1, 0, 0, 2, 1, 3, 3], [0, 2, 3, 6]
    g = torch.Generator(device="cuda").manual_seed(4)
    rand = lambda n: torch.randn(n, hidden, generator=g, device="cuda").half()  # noqa: E731
    xp, xt, xn = rand(sum(prompts)), rand(R * len(parents)), rand(R)
    tree, chain = (AttentionBlock(Wqkv, Wo, hidden, heads, kv_heads, D, R, 40, 16, page=16, q8=q8) for _ in range(2))
    for b in (tree, chain):
        b.step(xp, new(*prompts))
    mask = torch.from_numpy(np.concatenate([tree_mask(parents)] * R)).cuda()
    y, maps = tree.step(xt, new(*[len(parents)] * R), tree=mask)
    assert maps.pos.view(R, -1).tolist() == [[p + d for d in (0, 1, 1, 2, 2, 3, 3)] for p in prompts]
    for r in range(R):
        tree.keep(r, maps, path)
    assert torch.equal(tree.lens, new(*[p + len(path) for p in prompts]))
    # The two runs differ by which kernel takes the products (fp16 partial sums at
    # one token, fp32 at many: 2e-3 of the sum of magnitudes each, far less here)
    # and, through it, by roundings of the cached rows.
    tol = 1e-2
    for node in path:
        at = torch.arange(R, device="cuda") * len(parents) + node
        y1, _ = chain.step(xt[at], new(*[1] * R))
        assert float((y1 - y[at]).norm() / y1.norm()) < tol
    a, _ = tree.step(xn, new(*[1] * R))
    b, _ = chain.step(xn, new(*[1] * R))
    assert float((a - b).norm() / b.norm()) < tol
    assert q.qmv_device_status() == 0


def test_pages_append_graph_and_pdl_agree(q):
    """Maps and cache write: the same bits eagerly, without dependent launch,
    and replayed from a graph on a side stream."""
    rs = np.random.RandomState(1)
    R, page, heads, hk, D = 5, 16, 4, 2, 128
    dev = lambda a: torch.from_numpy(np.asarray(a)).cuda()  # noqa: E731
    lens, news = rs.randint(0, 40, R).astype(np.int32), rs.randint(1, 9, R).astype(np.int32)
    have = -(-lens // page)
    table = np.full((R, 4), -1, dtype=np.int32)
    for r in range(R):
        table[r, :have[r]] = 10 * r + np.arange(have[r])
    T = int(news.sum())
    ln, nn, tb, fr = dev(lens), dev(news), dev(table), dev(np.arange(60, 80, dtype=np.int32))
    x = torch.randn(T, (heads + 2 * hk) * D, device="cuda")
    ang = torch.rand(100, 64, device="cuda") * 6
    cos, sin = ang.cos(), ang.sin()

    def call(cache, stream=None):
        p = q.qmv_kv_pages(ln, nn, fr, tb, page, T, stream=stream)
        return p, q.qmv_kv_append(x, cache, p.slots, heads, pos=p.pos, cos=cos, sin=sin, stream=stream)

    for dt in (torch.float16, torch.int8):
        caches = [q.qmv_kv_cache(80, hk, page, D, dt) for _ in range(3)]
        torch.cuda.synchronize()
        first = call(caches[0])
        q.qmv_set_pdl(False)
        try:
            off = call(caches[1])
        finally:
            q.qmv_set_pdl(True)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            with torch.cuda.graph(g, stream=s):
                replayed = call(caches[2], stream=s)
        g.replay()
        torch.cuda.synchronize()
        for other, c in ((off, caches[1]), (replayed, caches[2])):
            assert all(torch.equal(a, b) for a, b in zip(first[0], other[0])) and torch.equal(first[1], other[1])
            for name in ("k", "v", "k_scale", "v_scale"):
                a, b = getattr(caches[0], name), getattr(c, name)
                assert (a is None and b is None) or torch.equal(a, b)
        assert q.qmv_device_status() == 0
