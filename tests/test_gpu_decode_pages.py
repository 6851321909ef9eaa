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
