"""Page and slot maps and the rotary cache write on the GPU, against plain
64-bit forms: whole numbers equal, stored rows within their rounding."""
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


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run_pages(q, lens, news, free, table, page, tokens, head=None, tree=None, **kw):
    t = dev(table)
    p = q.qmv_kv_pages(dev(lens), dev(news), dev(free), t, page, tokens,
                       head=None if head is None else dev(np.array([head], dtype=np.int32)),
                       tree=None if tree is None else dev(tree), **kw)
    got = {k: getattr(p, k).cpu().numpy() for k in p._fields}
    got["table"] = t.cpu().numpy()
    return got


def setup(R, len_hi, new_hi, page, seed, zero_new=True):
    rs = np.random.RandomState(seed)
    lens = rs.randint(0, len_hi + 1, R).astype(np.int32)
    news = rs.randint(0 if zero_new else 1, new_hi + 1, R).astype(np.int32)
    have = -(-lens // page)
    need = -(-(lens + news) // page)
    ids = rs.permutation(int(need.sum()) + 40).astype(np.int32)
    table = np.full((R, int(need.max()) + 1 if R else 1), -7, dtype=np.int32)
    at = 0
    for r in range(R):
        table[r, :have[r]] = ids[at:at + have[r]]
        at += have[r]
    return lens, news, ids[at:].copy(), table


@pytest.mark.parametrize("R,len_hi,new_hi,page,pad,head", [
    (1, 0, 1, 16, 0, None), (1, 1000, 8, 16, 0, 3), (7, 100, 33, 32, 5, 0), (64, 500, 1, 64, 0, 2),
    (1024, 90, 9, 16, 1000, 1), (1025, 90, 5, 16, 0, None), (2600, 40, 3, 16, 17, 4), (3, 5000, 4000, 256, 3000, 0),
    (33, 300, 0, 16, 9, 0),
])
def test_pages(q, R, len_hi, new_hi, page, pad, head):
    lens, news, free, table = setup(R, len_hi, new_hi, page, 10 * R + page)
    tokens = int(news.sum()) + pad
    got = run_pages(q, lens, news, free, table, page, tokens, head)
    want = ref.pages(lens, news, free, table, page, tokens, head or 0)
    for k, w in want.items():
        assert np.array_equal(got[k], np.asarray(w, dtype=np.int32)), k
    assert q.qmv_device_status() == 0


@pytest.mark.parametrize("words", [1, 2, 5])
def test_pages_tree_depths(q, words):
    lens, news, free, table = setup(20, 200, 32 * words, 16, words, zero_new=False)
    tree = ref.random_trees(list(news), words, np.random.RandomState(words))
    tree[3] = 0                        # sees nothing: depth not below zero
    tree[5] = -1                       # every bit, past the last node too
    got = run_pages(q, lens, news, free, table, 16, int(news.sum()), tree=tree)
    want = ref.pages(lens, news, free, table, 16, int(news.sum()), tree=tree)
    for k, w in want.items():
        assert np.array_equal(got[k], np.asarray(w, dtype=np.int32)), k
    assert q.qmv_device_status() == 0


def test_pages_no_requests(q):
    e = np.zeros(0, dtype=np.int32)
    got = run_pages(q, e, e, np.arange(4, dtype=np.int32), np.zeros((0, 3), dtype=np.int32), 16, 6, head=2)
    assert got["start"].tolist() == [0] and got["head"].tolist() == [2]
    assert got["slots"].tolist() == [-1] * 6 and got["request"].tolist() == [-1] * 6
    assert q.qmv_device_status() == 0


def test_pages_short_list_table_and_outputs(q):
    lens, news, free, table = setup(40, 60, 50, 16, 5, zero_new=False)
    tokens = int(news.sum())
    for kw in ({"free": free[:11]}, {"table": table[:, :3]}, {"tokens": tokens - 77}, {"tokens": 0}):
        a = {"free": free, "table": table, "tokens": tokens, **kw}
        lens_, news_ = lens, news
        if "table" in kw:
            lens_ = np.minimum(lens, 40)
        got = run_pages(q, lens_, news_, a["free"], a["table"], 16, a["tokens"])
        want = ref.pages(lens_, news_, a["free"], a["table"], 16, a["tokens"])
        for k, w in want.items():
            assert np.array_equal(got[k], np.asarray(w, dtype=np.int32)), (list(kw), k)
        assert q.qmv_device_status() == q.QMV_DEV_NO_PAGES, kw
    assert q.qmv_device_status() == 0


def test_pages_bad_ids_and_lengths(q):
    lens, news, free, table = setup(6, 60, 20, 16, 9, zero_new=False)
    lens[:] = 40
    table[:, :3] = np.arange(18).reshape(6, 3)
    free = np.arange(18, 58, dtype=np.int32)
    table[2, 2] = 1 << 20              # an old page outside the cache: its slots, no others
    got = run_pages(q, lens, news, free, table, 16, int(news.sum()), n_pages=100)
    want = ref.pages(lens, news, free, table, 16, int(news.sum()))
    at, s = np.asarray(want["start"]), np.asarray(want["slots"])
    for t in range(at[2], at[3]):
        if (40 + t - at[2]) // 16 == 2:
            s[t] = -1
    assert np.array_equal(got["slots"], s)
    assert q.qmv_device_status() == q.QMV_DEV_BAD_PAGE
    news[1], lens[4] = -3, -1
    table[2, 2] = 90
    got = run_pages(q, lens, news, free, table, 16, int(news.sum()) + 60, n_pages=100)
    n2 = news.copy()
    n2[[1, 4]] = 0
    l2 = np.maximum(lens, 0)
    want = ref.pages(l2, n2, free, table, 16, int(news.sum()) + 60)
    for k, w in want.items():
        assert np.array_equal(got[k], np.asarray(w, dtype=np.int32)), k
    assert q.qmv_device_status() == q.QMV_DEV_BAD_LENGTH


# -- rotary cache write ---------------------------------------------------------------

def make_cache(q, n_pages, hk, page, D, q8, together=False, fill=0.25):
    if q8:
        c = q.qmv_kv_cache(n_pages, hk, page, D, torch.int8)
        for t in (c.k, c.v):
            t.fill_(3)
        for t in (c.k_scale, c.v_scale):
            t.fill_(fill)
        return c
    if together:                       # k and v page by page in one buffer
        both = torch.full((n_pages, 2, hk, page, D), fill, dtype=torch.float16, device="cuda")
        return q.KvCache(both[:, 0], both[:, 1])
    c = q.qmv_kv_cache(n_pages, hk, page, D)
    c.k.fill_(fill)
    c.v.fill_(fill)
    return c


@pytest.mark.parametrize("D,heads,hk", [(128, 32, 8), (64, 64, 8), (128, 5, 1), (64, 3, 3), (128, 0, 2)])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("rot,inter,T", [("D", False, 1), ("D", True, 37), (0, False, 130), ("D/2", False, 9),
                                         (24, False, 33), (40, True, 8)])
def test_append(q, D, heads, hk, f32, q8, rot, inter, T):
    rot = {"D": D, "D/2": D // 2}.get(rot, rot)
    page, n_pages, n_pos = 16, T // 16 + 4, 300
    rs = np.random.RandomState(D + heads + T)
    wide = (heads + 2 * hk) * D
    x = (rs.randn(T, wide + 8) * 2).astype(np.float32 if f32 else np.float16)
    x[T // 2, (heads + hk) * D:(heads + hk + 1) * D] = 0       # an all-zero value row
    slots = rs.permutation(n_pages * page)[:T].astype(np.int32)
    if T > 5:
        slots[4] = -1
    pos = rs.randint(0, n_pos, T).astype(np.int32)
    ang = np.arange(n_pos)[:, None] * 1000.0 ** (-np.arange(max(1, rot // 2)) / max(1, rot // 2))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    c = make_cache(q, n_pages, hk, page, D, q8, together=T == 37)
    xd = dev(x)[:, :wide]                                      # rows wider apart than their values
    kw = dict(pos=dev(pos), cos=dev(cos), sin=dev(sin), interleaved=inter) if rot else {}
    qo = q.qmv_kv_append(xd, c, dev(slots), heads, **kw).cpu().numpy().astype(np.float64)
    assert q.qmv_device_status() == 0
    y = x[:, :wide].astype(np.float64).reshape(T, -1, D)
    mag = np.abs(y)
    if rot:
        cs, sn = cos.astype(np.float64)[pos][:, None], sin.astype(np.float64)[pos][:, None]
        turned, part = y[:, :heads + hk], mag[:, :heads + hk]
        y = np.concatenate([ref.rotate(turned, rot, inter, cs, sn), y[:, heads + hk:]], 1)
        mag = np.concatenate([ref.rotate(part, rot, inter, np.abs(cs), -np.abs(sn)), mag[:, heads + hk:]], 1)
        mag = np.maximum(np.abs(mag), np.abs(y)) + np.abs(x[:, :wide].astype(np.float64)).max()
    err32 = 3 * 2.0 ** -24 * mag if rot else 0 * mag           # two products and a sum in fp32
    assert np.all(np.abs(qo - y[:, :heads]) <= (2.0 ** -11 * np.abs(y) + err32 + 2.0 ** -25)[:, :heads])
    for name, first in (("k", heads), ("v", heads + hk)):
        pool = getattr(c, name).cpu().numpy().astype(np.float64)
        fill = np.full_like(pool, 0.25 * 3 if q8 else 0.25)
        if q8:
            codes, d = pool, getattr(c, name + "_scale").cpu().numpy().astype(np.float64)
            pool = pool * d[..., None]
        want, tol = fill, np.zeros_like(fill)
        for t in range(T):
            if slots[t] < 0:
                continue
            at = (slots[t] // page, slice(None), slots[t] % page)
            want[at] = y[t, first:first + hk]
            e = err32[t, first:first + hk]
            if q8:
                amax = np.abs(want[at]).max(-1, keepdims=True)
                # half a code, and the fp32 roundings of d, 1 / d and the product (127 codes of 3 roundings)
                tol[at] = amax / 127 * (0.5 + 127 * 4 * 2.0 ** -24) + 2 * e.max(-1, keepdims=True)
                assert np.abs(codes[at]).max() <= 127
                assert np.all(np.abs(d[at] - amax[..., 0] / 127) <= 2.0 ** -23 * d[at] + e.max(-1) / 127)
            else:
                tol[at] = 2.0 ** -11 * np.abs(want[at]) + e + 2.0 ** -25
        assert np.all(np.abs(pool - want) <= tol), name
    if T > 5:
        assert np.isfinite(qo).all()


def test_append_bad_slots_and_positions(q):
    c = make_cache(q, 4, 2, 16, 64, False)
    before = c.k.clone()
    x = torch.randn(3, 6 * 64, device="cuda")
    cos = torch.ones(10, 32, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    q.qmv_kv_append(x, c, i32(64, -2, 1 << 30), 2, pos=i32(0, 1, 2), cos=cos, sin=cos)
    assert q.qmv_device_status() == q.QMV_DEV_BAD_PAGE and torch.equal(c.k, before)
    out = q.qmv_kv_append(x, c, i32(0, 1, 2), 2, pos=i32(10, 3, -1), cos=cos, sin=cos)
    assert q.qmv_device_status() == q.QMV_DEV_BAD_LENGTH
    assert out[0].isnan().all() and out[2].isnan().all() and out[1].isfinite().all()
    assert torch.equal(c.k[0, :, 0], before[0, :, 0]) and not torch.equal(c.k[0, :, 1], before[0, :, 1])


def test_append_past_two_gigabytes(q):
    """A slot whose byte and element offsets pass 32 bits."""
    page, hk, D = 64, 8, 128
    n_pages = (1 << 32) // (page * hk * D) + 3
    c = q.KvCache(*(torch.empty((n_pages, hk, page, D), dtype=torch.float16, device="cuda") for _ in range(2)))
    x = torch.randn(2, (2 + 2 * hk) * D, device="cuda")
    last = n_pages * page - 1
    q.qmv_kv_append(x, c, torch.tensor([last, 5], dtype=torch.int32, device="cuda"), 2)
    assert torch.equal(c.k[n_pages - 1, :, page - 1], x[0, 2 * D:(2 + hk) * D].view(hk, D).half())
    assert torch.equal(c.v[0, :, 5], x[1, (2 + hk) * D:].view(hk, D).half())
    assert q.qmv_device_status() == 0


def test_refusals(q):
    c = q.qmv_kv_cache(4, 2, 16, 64)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.zeros(3, 6 * 64, device="cuda")
    with pytest.raises(TypeError):
        q.qmv_kv_pages(i32(2).long(), i32(2), i32(4), i32(2, 3), 16, 4)
    with pytest.raises(ValueError):
        q.qmv_kv_pages(i32(2), i32(3), i32(4), i32(2, 3), 16, 4)
    with pytest.raises(q.QmvError):
        q.qmv_kv_pages(i32(2), i32(2), i32(4), i32(2, 3), 24, 4)      # page not a power of two
    with pytest.raises(ValueError):
        q.qmv_kv_pages(i32(2), i32(2), i32(4), i32(2, 3), 16, 4, tree=i32(3, 1))
    with pytest.raises(TypeError):
        q.qmv_kv_pages(i32(2).cpu(), i32(2), i32(4), i32(2, 3), 16, 4)
    with pytest.raises(ValueError):
        q.qmv_kv_append(x, c, i32(2), 2)                               # slots of another length
    with pytest.raises(ValueError):
        q.qmv_kv_append(x, c, i32(3), 3)                               # row of another width
    with pytest.raises(TypeError):
        q.qmv_kv_append(x.double(), c, i32(3), 2)
    with pytest.raises(ValueError):
        q.qmv_kv_append(x, c, i32(3), 2, cos=torch.ones(4, 32, device="cuda"), sin=torch.ones(4, 32, device="cuda"))
    with pytest.raises(q.QmvError):                                    # rot not a multiple of 8
        q.qmv_kv_append(x, c, i32(3), 2, pos=i32(3), cos=torch.ones(4, 6, device="cuda"),
                        sin=torch.ones(4, 6, device="cuda"))
    with pytest.raises(q.QmvError):                                    # rows that are not 16-byte aligned
        q.qmv_kv_append(torch.zeros(3, 6 * 64 + 2, device="cuda")[:, :6 * 64], c, i32(3), 2)
    with pytest.raises(ValueError):
        q.KvCache(c.k, c.v.transpose(1, 2))
    with pytest.raises(ValueError):
        q.KvCache(c.k.to(torch.int8), c.v.to(torch.int8))              # no scales
    with pytest.raises(TypeError):
        q.KvCache(c.k.float(), c.v.float())
    assert q.qmv_device_status() == 0


def test_cache_objects_cannot_be_changed_and_follow_their_storage(q):
    """A KvCache refuses other tensors; its calls use its tensors' memory as it
    is at the call, also after the storage was given up and taken again."""
    c = q.qmv_kv_cache(4, 2, 16, 64)
    for name in ("k", "kind", "page_stride"):
        with pytest.raises(AttributeError):
            setattr(c, name, getattr(c, name))
    qkv = torch.randn(3, (4 + 2 * 2) * 64, device="cuda")
    slots = torch.tensor([0, 17, 63], dtype=torch.int32, device="cuda")
    size, old = c.k.untyped_storage().nbytes(), c.k.data_ptr()
    c.k.untyped_storage().resize_(0)
    keep = torch.empty(size, dtype=torch.uint8, device="cuda")     # takes the old place
    c.k.untyped_storage().resize_(size)
    keep.zero_()
    q.qmv_kv_append(qkv, c, slots, 4)
    at = [(int(s) // 16, int(s) % 16) for s in slots]
    for t, (page, row) in enumerate(at):
        assert torch.equal(c.k[page, :, row], qkv[t, 256:384].half().view(2, 64))
    assert c.k.data_ptr() == old or not keep.any()
