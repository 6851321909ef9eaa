"""Attention over the paged cache: seeded random shapes over every layout, many
small requests, workspaces with anything in them, and calls side by side."""
import threading

import numpy as np
import pytest

from tests import kv_reference as ref
from tests.test_gpu_tree_attn import call, check, dev

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


@pytest.mark.parametrize("seed", range(40))
def test_random_shapes(q, ws, seed):
    rs = np.random.RandomState(1000 + seed)
    D = int(rs.choice([64, 128]))
    hk = int(rs.choice([1, 2, 3, 8]))
    heads = hk * int(rs.choice([1, 2, 4, 5, 8, 16]))
    R = int(rs.choice([1, 1, 2, 5, 13]))
    top = int(np.exp(rs.uniform(0, np.log(2000 if R < 5 else 300))))
    new = int(np.exp(rs.uniform(0, np.log(100 if heads < 20 else 40))))
    lens = [int(v) for v in rs.randint(0, top + 1, R)]
    news = [int(v) for v in rs.randint(0, new + 1, R)]
    news[rs.randint(R)] = new
    page = int(rs.choice([16, 32, 64, 128, 256]))
    tree = "random" if rs.rand() < 0.5 else None
    check(q, ref.problem(lens, news, heads, hk, D, page, q8=bool(rs.rand() < 0.5), tree=tree, seed=seed,
                         spread=float(rs.choice([0.3, 1.0, 3.0]))), ws)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("R,new,heads,hk", [(700, 1, 4, 1), (450, 5, 8, 1), (1100, 2, 2, 2)])
def test_more_requests_than_threads(q, ws, R, new, heads, hk, q8):
    rs = np.random.RandomState(R)
    lens = [int(v) for v in rs.randint(0, 60, R)]
    lens[R - 1], lens[R // 2] = 900, 0
    check(q, ref.problem(lens, [new] * R, heads, hk, 64, 16, q8=q8, seed=R), ws)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("L,T", [(5000, 1), (3000, 9), (2000, 40), (900, 90)])
def test_workspace_holds_anything(q, L, T, q8):
    """The workspace's contents do not matter, and calls repeat bit for bit."""
    prob = ref.problem([L, 50], [T, T], 8, 2, 128, 32, q8=q8, tree="random", seed=T)
    ws = q.qmv_tree_attn_workspace()
    ws.fill_(255)
    a = call(q, prob, ws)
    ws.fill_(1)
    b = call(q, prob, ws)
    assert torch.equal(a, b)
    check(q, prob, ws)


def test_calls_on_several_streams(q):
    """Four host threads, each with its stream and workspace, calls of different
    kernels at once: every one gives what it gives alone."""
    probs = [ref.problem([4000], [1], 8, 2, 128, 32, seed=1), ref.problem([3000, 100], [8, 8], 8, 2, 64, 16, q8=True, seed=2),
             ref.problem([1500], [60], 8, 2, 128, 64, seed=3), ref.problem([800, 900], [40, 1], 16, 2, 64, 16, q8=True, seed=4)]
    args = []
    for p in probs:
        c = q.KvCache(*(dev(p[n]) for n in ("k", "v", "k_scale", "v_scale")))
        args.append((dev(p["q"]), c, dev(p["table"]), dev(p["start"]), dev(p["kv_len"])))
    alone = [q.qmv_tree_attn(*a, workspace=q.qmv_tree_attn_workspace()) for a in args]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def work(i):
        try:
            s, ws = torch.cuda.Stream(), q.qmv_tree_attn_workspace()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                for _ in range(20):
                    got[i] = q.qmv_tree_attn(*args[i], workspace=ws)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for a, b in zip(alone, got):
        assert torch.equal(a, b)
    assert q.qmv_device_status() == 0


def test_a_workspace_is_made_where_none_is_given(q):
    prob = ref.problem([700], [3], 8, 2, 64, 16, seed=8)
    check(q, prob, None)


@pytest.mark.parametrize("scale", [0.0, 0.3, -0.3, 1.0])
@pytest.mark.parametrize("heads,D,T", [(4, 64, 6), (4, 128, 3), (16, 64, 20), (16, 128, 40)])
def test_row_scales_of_either_sign_and_zero(q, ws, heads, D, T, scale):
    """8-bit rows whose scales are negative, zero (over codes that are not),
    least normal or subnormal: hidden places stay hidden, the others count."""
    prob = ref.problem([70, 3], [T, 5], heads, 2, D, 16, q8=True, tree="random", seed=T)
    rs = np.random.RandomState(1)
    for name in ("k_scale", "v_scale"):
        arr = prob[name]
        arr *= np.where(rs.rand(*arr.shape) < 0.4, -1.0, 1.0).astype(np.float32)
        for value in (0.0, -0.0, 2.0 ** -126, 2.0 ** -149):
            arr[rs.rand(*arr.shape) < 0.06] = value
    check(q, prob, ws, scale=scale)
    check(q, {**prob, "tree": None}, ws, scale=scale)
