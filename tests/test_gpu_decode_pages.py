"""Pages through hundreds of steps that draft a tree of tokens and keep a part of
it: none is lost, none is in two places."""
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
    yield m
    torch.cuda.synchronize()


def small_block(requests, n_pages, width, page):
    from weight_quantized_decode_gb300.decode_block import AttentionBlock
    hidden, heads, kv_heads, D = 256, 4, 2, 64
    Wqkv = torch.from_numpy(synth.q4_0_weights((heads + 2 * kv_heads) * D, hidden, 1)).cuda()
    Wo = torch.from_numpy(synth.q4_0_weights(hidden, heads * D, 2)).cuda()
    return AttentionBlock(Wqkv, Wo, hidden, heads, kv_heads, D, requests, n_pages, width, page=page), hidden


@pytest.mark.parametrize("page", [16, 32])
def test_pages_of_rejected_nodes_are_not_lost(q, page):
    """Two requests, 250 steps of eight nodes of which one to four stay, on a
    cache that holds just what the requests come to hold."""
    from weight_quantized_decode_gb300.decode_block import tree_mask
    rs = np.random.RandomState(page)
    prompts, nodes, steps = [37, 5], 8, 250
    kept = rs.randint(1, 5, (steps, 2))
    most = [max(p + int(kept[:i, r].sum()) + nodes for i in range(steps)) for r, p in enumerate(prompts)]
    n_pages = sum(-(-m // page) for m in most)
    block, hidden = small_block(2, n_pages, max(-(-m // page) for m in most), page)
    new = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    mask = torch.from_numpy(np.concatenate([tree_mask(list(range(-1, nodes - 1)))] * 2)).cuda()
    x = torch.randn(max(sum(prompts), 2 * nodes), hidden, device="cuda").half()
    block.step(x[:sum(prompts)], new(*prompts))
    for i in range(steps):
        y, maps = block.step(x[:2 * nodes], new(nodes, nodes), tree=mask)
        if i % 50 == 49 or i == steps - 1:
            table = block.table.cpu().numpy()
            held = table[table >= 0]
            assert len(np.unique(held)) == len(held) == int(block.head), i
            assert (maps.slots >= 0).all() and torch.isfinite(y).all(), i
        for r in range(2):
            block.keep(r, maps, list(range(kept[i, r])))
    assert block.lens.tolist() == [p + int(kept[:, r].sum()) for r, p in enumerate(prompts)]
    assert int(block.head) == n_pages
    assert q.qmv_device_status() == 0


def plain_pages(lens, news, free, table, page, tokens, head, held):
    """qmv_kv_pages with `held`, one request after another (enough pages and room)."""
    table, slots, kept, at, used = table.copy(), [], [], head, 0
    for r, (a, n) in enumerate(zip(lens, news)):
        have = max(int(held[r]), -(-int(a) // page))
        need = -(-(int(a) + int(n)) // page)
        for j in range(have, need):
            table[r, j] = free[at]
            at += 1
        kept.append(max(have, need))
        slots += [table[r, (int(a) + i) // page] * page + (int(a) + i) % page for i in range(int(n))]
    return table, slots + [-1] * (tokens - len(slots)), at, kept


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


@pytest.mark.parametrize("R", [1, 5, 1024, 1500])
def test_pages_past_a_length_are_used_again(q, R):
    rs = np.random.RandomState(R)
    page, width, head = 16, 12, 3
    lens, news = rs.randint(0, 90, R), rs.randint(0, 60, R)
    filled = -(-lens // page)
    held = np.minimum(filled + rs.randint(0, 4, R) * (rs.rand(R) < 0.6), width)
    held[rs.rand(R) < 0.2] = 0                         # fewer than the length fills: the length counts
    have = np.maximum(held, filled)
    ids = rs.permutation(int(have.sum()) + 6 * R + head).astype(np.int32)
    table, at = np.full((R, width), -1, dtype=np.int32), 0
    for r in range(R):
        table[r, :have[r]] = ids[at:at + have[r]]
        at += have[r]
    free, tokens = ids[at:], int(news.sum()) + 7
    want = plain_pages(lens, news, free, table, page, tokens, head, held)
    td, args = dev(table), (dev(lens), dev(news), dev(free))
    for _ in range(2):                                 # the same inputs: the same outputs
        p = q.qmv_kv_pages(*args, td, page, tokens, head=dev([head]), held=dev(held))
        assert np.array_equal(td.cpu().numpy(), want[0]) and p.slots.tolist() == want[1]
        assert int(p.head) == want[2] and p.held.tolist() == want[3]
        assert p.kv_len.tolist() == (lens + news).tolist()
    plain = q.qmv_kv_pages(*args, dev(table), page, tokens, head=dev([head]))
    none = q.qmv_kv_pages(*args, dev(table), page, tokens, head=dev([head]), held=dev(np.zeros(R)))
    for name in plain._fields:                         # nothing held: what the length fills
        assert torch.equal(getattr(plain, name), getattr(none, name)), name
    assert none.held.tolist() == np.maximum(filled, -(-(lens + news) // page)).tolist()
    assert q.qmv_device_status() == 0


def test_held_counts_pages_that_there_were(q):
    """A list or a row that ends counts the pages there were; counts out of range are reported."""
    lens, news, table = dev([20, 0]), dev([60, 40]), np.array([[7, 8, -1, -1], [-1, -1, -1, -1]])
    p = q.qmv_kv_pages(lens, news, dev([1, 2, 3, 4, 5]), dev(table), 16, 100, held=dev([2, 0]))
    assert p.held.tolist() == [4, 3] and int(p.head) == 5 and q.qmv_device_status() == q.QMV_DEV_NO_PAGES
    p = q.qmv_kv_pages(lens, news, dev([1, 2, 3]), dev(table), 16, 100, held=dev([2, 0]))
    assert p.held.tolist() == [4, 1] and int(p.head) == 3 and q.qmv_device_status() == q.QMV_DEV_NO_PAGES
    t = dev(table)
    p = q.qmv_kv_pages(lens, dev([0, 0]), dev([1]), t, 16, 0, held=dev([-1, 9]))
    assert p.held.tolist() == [2, 4] and np.array_equal(t.cpu().numpy(), table)
    assert q.qmv_device_status() == q.QMV_DEV_BAD_LENGTH
    with pytest.raises(ValueError):
        q.qmv_kv_pages(lens, news, dev([1]), dev(table), 16, 100, held=dev([1]))
    with pytest.raises(TypeError):
        q.qmv_kv_pages(lens, news, dev([1]), dev(table), 16, 100, held=dev([1, 1]).float())


def test_nothing_is_kept_of_a_step_without_pages(q):
    """A step whose free list ran out left tokens without a slot: keep refuses, and no
    row of the cache changes (a slot of -1 would be the last page's last row)."""
    from weight_quantized_decode_gb300.decode_block import tree_mask
    block, hidden = small_block(1, 2, 4, 16)
    mask = torch.from_numpy(tree_mask([-1, 0, 0, 2])).cuda()
    x = torch.randn(31, hidden, device="cuda").half()
    block.step(x, dev([31]))
    _, maps = block.step(x[:4], dev([4]), tree=mask)
    assert (maps.slots < 0).any() and q.qmv_device_status() != 0
    before = block.cache.k.clone(), block.cache.v.clone(), block.lens.clone()
    with pytest.raises(RuntimeError):
        block.keep(0, maps, [0, 2, 3])
    for a, b in zip(before, (block.cache.k, block.cache.v, block.lens)):
        assert torch.equal(a, b)
