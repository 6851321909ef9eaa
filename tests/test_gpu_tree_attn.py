"""Attention over the paged cache on the GPU against the plain 64-bit form,
per output, with the allowance tests/kv_reference.py derives."""
import numpy as np
import pytest

from tests import kv_reference as ref

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


@pytest.fixture(scope="module")
def ws(q):
    return q.qmv_tree_attn_workspace()


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def call(q, prob, ws, scale=None, out=None, qd=None, cache=None, stream=None):
    c = cache or q.KvCache(*(dev(prob[n]) for n in ("k", "v", "k_scale", "v_scale")))
    return q.qmv_tree_attn(dev(prob["q"]) if qd is None else qd, c, dev(prob["table"]), dev(prob["start"]),
                           dev(prob["kv_len"]), tree=dev(prob["tree"]), scale=scale, out=out, workspace=ws,
                           stream=stream)


def check(q, prob, ws, scale=None, **kw):
    got = call(q, prob, ws, scale, **kw).cpu().numpy().astype(np.float64)
    want, allow = ref.attention(prob, prob["q"].shape[2] ** -0.5 if scale is None else scale)
    err = np.abs(got - want)
    assert np.isfinite(got).all()
    assert np.all(err <= allow), (float((err / allow).max()), np.unravel_index((err / allow).argmax(), err.shape))
    assert q.qmv_device_status() == 0
    return got


LAYOUTS = [(8, 8, 128), (32, 8, 128), (7, 1, 64), (64, 8, 64), (12, 4, 64), (20, 1, 128), (3, 3, 64), (40, 2, 128)]


@pytest.mark.parametrize("heads,hk,D", LAYOUTS)
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("lens,news,page", [
    ((0,), (1,), 16), ((1,), (1,), 16), ((15, 16, 17), (1, 1, 1), 16), ((300,), (1,), 32),
    ((0, 63, 130), (5, 9, 3), 64), ((700,), (8,), 128), ((31, 0, 257, 90), (0, 2, 33, 0), 16), ((129,), (70,), 256),
])
def test_chain(q, ws, heads, hk, D, q8, lens, news, page):
    check(q, ref.problem(list(lens), list(news), heads, hk, D, page, q8=q8, seed=len(lens) + heads), ws)


@pytest.mark.parametrize("heads,hk,D", LAYOUTS)
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("lens,news,page", [
    ((100,), (8,), 16), ((0,), (31,), 16), ((5, 200, 64), (64, 1, 17), 32), ((1000, 3), (24, 40), 64)])
def test_tree(q, ws, heads, hk, D, q8, lens, news, page):
    check(q, ref.problem(list(lens), list(news), heads, hk, D, page, q8=q8, tree="random", seed=heads), ws)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("L,T", [(4000, 1), (4097, 3), (9001, 16), (2500, 130), (20011, 2), (600, 300)])
def test_long(q, ws, q8, D, L, T):
    """Contexts that are split over many SMs and joined, few and many rows."""
    check(q, ref.problem([L], [T], 8, 2, D, 64, q8=q8, tree="random" if T == 16 else None, seed=L), ws)


def test_many_uneven_requests(q, ws):
    rs = np.random.RandomState(3)
    lens = [int(v) for v in rs.randint(0, 400, 150)]
    news = [int(v) for v in rs.randint(0, 4, 150)]
    lens[7], lens[90] = 6000, 3333
    check(q, ref.problem(lens, news, 4, 2, 128, 16, seed=3, width=500), ws)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("heads,D", [(4, 128), (16, 64)])
def test_masks(q, ws, q8, heads, D):
    """Rows that see nothing, everything, later nodes, or bits past the last
    node; masks with fewer words than nodes."""
    news = [40, 9, 70]
    for lens in ([0, 0, 0], [33, 100, 7]):
        tree = ref.random_trees(news, 3, np.random.RandomState(1))
        tree[[0, 5, 41]] = 0
        tree[[6, 44, 60]] = -1
        tree[7] = 1 << 30
        prob = ref.problem(lens, news, heads, 2, D, 16, q8=q8, tree=tree, seed=2)
        got = check(q, prob, ws)
        if lens[0] == 0:
            assert np.all(got[[0, 5, 41]] == 0)
        check(q, {**prob, "tree": np.ascontiguousarray(tree[:, :1])}, ws)     # nodes past 32 are unseen


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("heads,D,T", [(2, 64, 12), (16, 128, 40), (2, 128, 3)])
def test_unseen_values_do_not_reach_an_output(q, ws, q8, bad, heads, D, T):
    """NaN and infinities in stale rows, in unused pages and in tree nodes off
    a row's path: rows that do not see them keep their values."""
    prob = ref.problem([50, 10], [T, 2], heads, 2, D, 16, q8=q8, tree="random", seed=4, words=2)
    tree = prob["tree"]
    for name in ("k", "v"):
        arr = prob[name + "_scale"] if q8 else prob[name]
        used = prob["table"][prob["table"] >= 0]
        unused = np.setdiff1d(np.arange(arr.shape[0]), used)
        arr[unused] = bad
        for r in range(2):
            n = int(prob["kv_len"][r])
            if n % 16:
                arr[prob["table"][r, n // 16], :, n % 16:] = bad
    check(q, prob, ws)
    want, allow = ref.attention(prob, D ** -0.5)
    for node in (T - 1, 1):            # one node of the first request, its k or its v row
        for name in ("k", "v"):
            p2 = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in prob.items()}
            at = 50 + node
            arr = p2[name + "_scale"] if q8 else p2[name]
            arr[p2["table"][0, at // 16], :, at % 16] = bad
            got = call(q, p2, ws).cpu().numpy().astype(np.float64)
            off = [t for t in range(T + 2) if t >= T or not (int(tree[t, node // 32]) >> (node % 32) & 1)]
            assert np.all(np.abs(got[off] - want[off]) <= allow[off])
            on = [t for t in range(T) if t not in off]
            assert on
            if name == "v" and not (q8 and np.isinf(bad)):
                assert not np.isfinite(got[on]).any()


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0, 6.0])
def test_scales_and_large_scores(q, ws, q8, scale):
    """Flat, reversed and one-sided softmax (scores of hundreds)."""
    for lens, news in (([200, 9], [5, 17]), ([1500], [90])):
        check(q, ref.problem(lens, news, 6, 2, 64, 32, q8=q8, seed=11, spread=2.0), ws, scale=scale)


@pytest.mark.parametrize("T", [2, 70])
@pytest.mark.parametrize("up", [True, False])
def test_value_scales_of_every_size(q, ws, T, up):
    """8-bit rows whose scales rise or fall over many powers of two: nothing
    overflows the fp16 weights, and large rows keep their accuracy."""
    prob = ref.problem([300], [T], 4, 2, 64, 16, q8=True, seed=5)
    n = int(prob["kv_len"][0])
    e = np.linspace(-30, 40, n) if up else np.linspace(40, -30, n)
    for j in range(n):
        prob["v_scale"][prob["table"][0, j // 16], :, j % 16] = np.float32(2.0) ** np.float32(e[j])
    got = call(q, prob, ws).float()
    want, allow = ref.attention(prob, 0.125)
    g = got.cpu().numpy().astype(np.float64)
    # past fp16's largest value an output may be infinite; surely past it, it has to be one of the two
    may, must = np.abs(want) + allow >= 65504, np.abs(want) - allow >= 65520
    assert np.all(np.abs(g - want)[~may] <= allow[~may]) and np.all(np.abs(g[must]) >= 65504)
    assert not np.isnan(g).any()


def test_query_rows_apart_and_cache_in_one_buffer(q, ws):
    prob = ref.problem([77, 300], [3, 1], 8, 2, 128, 16, seed=6)
    T = 4
    wide = torch.randn(T, 12 * 128, device="cuda").half()
    qd = wide.as_strided((T, 8, 128), (12 * 128, 128, 1))
    qd.copy_(dev(prob["q"]))
    both = torch.full((prob["k"].shape[0], 2) + prob["k"].shape[1:], float("nan"), dtype=torch.float16, device="cuda")
    both[:, 0], both[:, 1] = dev(prob["k"]), dev(prob["v"])
    check(q, prob, ws, qd=qd, cache=q.KvCache(both[:, 0], both[:, 1]))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("heads,T", [(2, 2), (16, 20)])
def test_offsets_past_32_bits(q, ws, q8, heads, T):
    """Pages at the far end of a cache of more than 2^32 elements."""
    page, hk, D = 64, 2, 128
    n_pages = (1 << 32) // (page * hk * D) + 9
    prob = ref.problem([200], [T], heads, hk, D, page, q8=q8, seed=7, spare=0)
    far = torch.arange(n_pages - prob["k"].shape[0], n_pages, device="cuda")
    big = {}
    for n in ("k", "v", "k_scale", "v_scale"):
        if prob[n] is None:
            big[n] = None
            continue
        big[n] = torch.zeros((n_pages,) + prob[n].shape[1:], dtype=dev(prob[n][:1]).dtype, device="cuda")
        big[n][far] = dev(prob[n])
    p2 = {**prob, "table": prob["table"] + np.int32(n_pages - prob["k"].shape[0])}
    got = call(q, p2, ws, cache=q.KvCache(*big.values())).cpu().numpy().astype(np.float64)
    want, allow = ref.attention(prob, D ** -0.5)
    assert np.all(np.abs(got - want) <= allow) and q.qmv_device_status() == 0


@pytest.mark.parametrize("T", [2, 80])
def test_bad_pages_and_lengths(q, ws, T):
    """A request with a bad page id or length gives NaN and a status bit; the
    others keep their values."""
    good = ref.problem([60, 100, 30], [T, T, T], 4, 2, 64, 16, seed=8)
    want, allow = ref.attention(good, 0.125)
    for what, value in (("table", -1), ("table", 1 << 30), ("kv_len", T - 1), ("kv_len", -5), ("kv_len", 1 << 30)):
        p = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in good.items()}
        if what == "table":
            p["table"][1, 2] = value
        else:
            p["kv_len"][1] = value
        got = call(q, p, ws).cpu().numpy().astype(np.float64)
        assert np.isnan(got[T:2 * T]).all(), (what, value)
        ok = np.r_[0:T, 2 * T:3 * T]
        assert np.all(np.abs(got[ok] - want[ok]) <= allow[ok])
        assert q.qmv_device_status() == q.QMV_DEV_BAD_PAGE
    check(q, good, ws)


def test_rows_past_the_last_token_are_left(q, ws):
    prob = ref.problem([20, 5], [3, 2], 4, 2, 64, 16, seed=9)
    pad = {**prob, "q": np.concatenate([prob["q"], np.full((6, 4, 64), np.nan, np.float16)])}
    out = torch.full((11, 4, 64), 7.0, dtype=torch.float16, device="cuda")
    call(q, pad, ws, out=out)
    want, allow = ref.attention(prob, 0.125)
    assert np.all(np.abs(out[:5].cpu().numpy() - want) <= allow) and (out[5:] == 7).all()
    assert q.qmv_device_status() == 0


def test_nothing_to_do(q, ws):
    prob = ref.problem([20], [0], 4, 2, 64, 16, seed=9)
    assert call(q, prob, ws).shape == (0, 4, 64)
    assert q.qmv_device_status() == 0


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("lens,news,tree", [([5000], [1], None), ([300, 8000, 20], [8, 8, 3], "random"), ([900], [200], None)])
def test_eager_pdl_off_and_graph_agree(q, ws, q8, lens, news, tree):
    """The same bits eagerly, without dependent launch, from a side stream, and
    replayed from a graph, call after call on one workspace."""
    prob = ref.problem(lens, news, 8, 2, 128, 32, q8=q8, tree=tree, seed=10)
    c = q.KvCache(*(dev(prob[n]) for n in ("k", "v", "k_scale", "v_scale")))
    a = [dev(prob["q"]), c, dev(prob["table"]), dev(prob["start"]), dev(prob["kv_len"])]
    kw = dict(tree=dev(prob["tree"]), workspace=ws)
    torch.cuda.synchronize()
    first = q.qmv_tree_attn(*a, **kw)
    s = torch.cuda.Stream()
    q.qmv_set_pdl(False)
    try:
        off = q.qmv_tree_attn(*a, **kw)
    finally:
        q.qmv_set_pdl(True)
    torch.cuda.synchronize()
    side = q.qmv_tree_attn(*a, stream=s, **kw)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            y1 = q.qmv_tree_attn(*a, **kw)
            y2 = q.qmv_tree_attn(*a, **kw)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for y in (off, side, y1, y2):
        assert torch.equal(first, y)
    assert q.qmv_device_status() == 0


def test_a_decode_step_runs_as_one_graph(q, ws):
    """Maps, write and attention of two steps from device lengths alone."""
    rs = np.random.RandomState(12)
    heads, hk, D, page, R = 4, 2, 64, 16, 3
    c = q.qmv_kv_cache(40, hk, page, D)
    free = dev(rs.permutation(40).astype(np.int32))
    table = torch.full((R, 8), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(R, dtype=torch.int32, device="cuda")
    head = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept = [[] for _ in range(R)]
    for news in ([20, 3, 15], [1, 2, 30], [5, 0, 1]):
        x = torch.randn(sum(news), (heads + 2 * hk) * D, device="cuda")
        p = q.qmv_kv_pages(lens, dev(np.array(news, dtype=np.int32)), free, table, page, sum(news), head=head, n_pages=40)
        qo = q.qmv_kv_append(x, c, p.slots, heads)
        out = q.qmv_tree_attn(qo, c, table, p.start, p.kv_len, workspace=ws)
        lens, head = p.kv_len, p.head
        xs = x.half().double().cpu().numpy().reshape(-1, heads + 2 * hk, D)
        at = 0
        for r, n in enumerate(news):
            kept[r].append(xs[at:at + n, heads:])
            at += n
            if n == 0:
                continue
            kv = np.concatenate(kept[r])
            for i in range(n):
                seen = len(kv) - n + i + 1
                for h in range(heads):
                    s = kv[:seen, h // 2] @ xs[at - n + i, h] * 0.125
                    w = np.exp(s - s.max())
                    want = w @ kv[:seen, hk + h // 2] / w.sum()
                    a = w @ np.abs(kv[:seen, hk + h // 2]) / w.sum()
                    got = out[at - n + i, h].double().cpu().numpy()
                    assert np.all(np.abs(got - want) <= 2.0 ** -11 * np.abs(want) + 1.1 * 2.0 ** -11 * a + 2.0 ** -25)
    assert q.qmv_device_status() == 0


def test_refusals(q, ws):
    prob = ref.problem([20], [3], 4, 2, 64, 16, seed=13)
    c = q.KvCache(dev(prob["k"]), dev(prob["v"]))
    qd, t, s, n = (dev(prob[k]) for k in ("q", "table", "start", "kv_len"))
    ok = dict(workspace=ws)
    with pytest.raises(TypeError):
        q.qmv_tree_attn(qd.float(), c, t, s, n, **ok)
    with pytest.raises(TypeError):
        q.qmv_tree_attn(qd.cpu(), c, t, s, n, **ok)
    with pytest.raises(ValueError):
        q.qmv_tree_attn(qd[:, :, :32], c, t, s, n, **ok)
    with pytest.raises(ValueError):
        q.qmv_tree_attn(qd, c, t, s[:1], n, **ok)
    with pytest.raises(TypeError):
        q.qmv_tree_attn(qd, c, t.long(), s, n, **ok)
    with pytest.raises(ValueError):
        q.qmv_tree_attn(qd, c, t, s, n, tree=torch.zeros((2, 1), dtype=torch.int32, device="cuda"), **ok)
    with pytest.raises(q.QmvError):
        q.qmv_tree_attn(qd[:, :3], c, t, s, n, **ok)                   # heads not a multiple of kv heads
    with pytest.raises(q.QmvError):
        q.qmv_tree_attn(qd, c, t, s, n, scale=float("nan"), **ok)
    with pytest.raises(q.QmvError):                                    # a workspace that is too small
        q.qmv_tree_attn(qd, c, t, s, n, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    c48 = q.qmv_kv_cache(4, 2, 48, 64)
    with pytest.raises(q.QmvError):
        q.qmv_tree_attn(qd, c48, t, s, n, **ok)                        # page size
    c96 = q.qmv_kv_cache(4, 2, 16, 96)
    with pytest.raises(q.QmvError):
        q.qmv_tree_attn(torch.zeros(3, 4, 96, device="cuda").half(), c96, t, s, n, **ok)
    assert q.qmv_device_status() == 0
