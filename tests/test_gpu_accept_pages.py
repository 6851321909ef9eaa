"""The accepted path of a step that had no pages for some of its nodes: it ends where the rows end, and so does the
length."""
import numpy as np
import pytest

from tests import step_reference as ref
from tests.test_gpu_decode_drafts import VOCAB, decoder, ints
from tests.test_gpu_kv_pages import dev, q  # noqa: F401
from tests.test_gpu_tree_accept import host, problem

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def accept(tokens, sampled, start, kv_len, tree, slots):
    """The plain form's path, up to the first node without a row, or without a place to move its row to."""
    got = ref.accept(tokens, sampled, start, kv_len, tree)
    for r in range(len(kv_len)):
        lo, hi = int(start[r]), int(start[r + 1])
        n = 0
        while n < got["count"][r] and slots[lo + got["path"][lo + n]] >= 0 and slots[lo + n] >= 0:
            n += 1
        if n < got["count"][r]:
            got["next"][r] = int(sampled[lo + got["path"][lo + n - 1]]) if n else -1
            got["path"][lo + n:hi] = [-1] * (hi - lo - n)
            got["count"][r], got["lens"][r] = n, int(kv_len[r]) - (hi - lo) + n
    return got


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("nodes,words", [([1], 1), ([8], 1), ([33], 2), ([0, 5, 0, 31, 32, 33, 64, 1], 2), ([40] * 130, 2)])
def test_paths_end_with_the_rows(q, nodes, words, tree):  # noqa: F811
    """Slots that end somewhere in each request, and slots with holes.  (One token for all nodes, so that the lowest
    child is the accepted one with and without a row: rows end behind it or before it.)"""
    for seed in range(4):
        p = problem(nodes, words, seed, tree, 1)
        p["tokens"] = np.arange(len(p["tokens"]), dtype=np.int32)       # all different: one child at most is drawn
        rs = np.random.RandomState(seed)
        for r, n in enumerate(nodes):
            lo = int(p["start"][r])
            for c in range(n):
                row = [j for j in range(c + 1, n) if not tree and j == c + 1 or tree and j < 32 * words
                       and int(p["tree"][lo + j][c // 32]) >> (c % 32) & 1]
                p["sampled"][lo + c] = p["tokens"][lo + row[0]] if row and rs.rand() < 0.9 else 99999
        slots = rs.permutation(len(p["tokens"]) + 9)[:len(p["tokens"])].astype(np.int32)
        for r, n in enumerate(nodes):
            if seed < 3:
                slots[int(p["start"][r]) + rs.randint(0, n + 1):int(p["start"][r]) + n] = -1
            elif n:
                slots[int(p["start"][r]) + rs.randint(0, n)] = -1
        got = q.qmv_tree_accept(*(dev(p[n]) for n in ("tokens", "sampled", "start", "kv_len")),
                                tree=None if p["tree"] is None else dev(p["tree"]), slots=dev(slots))
        got = {n: getattr(got, n).tolist() for n in got._fields}
        assert got == accept(**p, slots=slots)
    with pytest.raises(ValueError):
        q.qmv_tree_accept(*(dev(p[n]) for n in ("tokens", "sampled", "start", "kv_len")), slots=dev(np.append(slots, slots)))
    assert q.qmv_device_status() == 0


PARENTS = [-1, 0, 0, 2]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("prompt,rows", [(29, 3), (30, 2), (31, 1), (32, 0), (28, 4)])
def test_a_verified_tree_without_pages(q, q8, prompt, rows):  # noqa: F811
    """Two pages of 16 and a prompt that leaves places for `rows` of four nodes, of which 0, 2, 3 are drawn: what has a
    row stays, in order, and the length ends behind it.  Then, with pages again, the request goes on as one that never
    ran short."""
    from weight_quantized_decode_gb300 import decode_block as b
    tree = dev(b.tree_mask(PARENTS))
    rs = np.random.RandomState(prompt)
    text = dev(rs.randint(0, VOCAB, prompt).astype(np.int32))
    tokens, sampled = ints(3, 4, 5, 6), ints(5, 0, 6, 7)
    short, full = decoder(1, q8, pages=4), decoder(1, q8, pages=4)
    pages, short.block.free = short.block.free, short.block.free[:2].clone()
    for d in (short, full):
        d.logits(text, ints(prompt))
    assert q.qmv_device_status() == 0
    maps = short.logits(tokens, ints(4), tree)[1]
    assert (maps.slots >= 0).sum() == rows
    assert bool(q.qmv_device_status() & q.QMV_DEV_NO_PAGES) == (rows < 4)
    before = host(short.block.cache)
    got = short.block.accept(tokens, sampled, maps, tree)
    count = {0: 0, 1: 1, 2: 1, 3: 2, 4: 3}[rows]
    kept = [0, 2, 3][:count]
    assert got.path.tolist() == kept + [-1] * (4 - count) and got.count.tolist() == [count]
    assert got.next.tolist() == [int(sampled[kept[-1]]) if kept else -1]
    assert got.lens.tolist() == short.block.lens.tolist() == [prompt + count]
    slots = maps.slots.cpu().numpy()
    for now, was in zip(host(short.block.cache), before):
        assert now is None or np.array_equal(now, ref.keep(was, slots, [0], kept, [count]))
    assert q.qmv_device_status() == 0
    # the same request in a cache with pages enough
    maps = full.logits(tokens, ints(4), tree)[1]
    if count:
        full.block.keep(0, maps, kept)
    else:
        full.block.lens = full.block.lens - 4
    short.block.free = pages
    a, w = (d.logits(ints(9, 8), ints(2))[0] for d in (short, full))
    assert short.block.lens.tolist() == full.block.lens.tolist()
    assert torch.isfinite(a).all() and (a - w).norm() <= 1e-2 * w.norm()
    assert q.qmv_device_status() == 0


def test_requests_beside_one_without_pages(q):  # noqa: F811
    """Three requests, of which the last finds no page: the others keep their whole paths; eager and captured alike."""
    from weight_quantized_decode_gb300 import decode_block as b
    tree = dev(np.concatenate([b.tree_mask(PARENTS)] * 3))
    d = decoder(3, pages=40)
    d.block.free = d.block.free[:3].clone()
    d.logits(dev(np.arange(36, dtype=np.int32)), ints(10, 10, 16))
    tokens, sampled = ints(*(3, 4, 5, 6) * 3), ints(*(5, 0, 6, 7) * 3)
    maps = d.logits(tokens, ints(4, 4, 4), tree)[1]
    q.qmv_device_status()
    g = torch.cuda.CUDAGraph()
    lens = d.block.lens
    with torch.cuda.graph(g):
        out = d.block.accept(tokens, sampled, maps, tree)
    d.block.lens = lens
    g.replay()
    torch.cuda.synchronize()
    assert out.path.tolist() == [0, 2, 3, -1] * 2 + [-1] * 4 and out.count.tolist() == [3, 3, 0]
    assert out.next.tolist() == [7, 7, -1] and out.lens.tolist() == [13, 13, 16]
    got = d.block.accept(tokens, sampled, maps, tree)
    for a, w in zip(got, out):
        assert torch.equal(a, w)
    assert q.qmv_device_status() == 0
