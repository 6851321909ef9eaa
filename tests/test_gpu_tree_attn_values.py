"""Attention over the paged cache with single values that stand out: what a
token does not see changes nothing, what it sees arrives once."""
import numpy as np
import pytest

from tests import kv_reference as ref
from tests.test_gpu_tree_attn import call, check

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


def copy(prob):
    return {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in prob.items()}


def seeing(prob, node, nodes):
    """Which of the first request's tokens see its node `node` (bool array)."""
    if prob["tree"] is None:
        return np.arange(nodes) >= node
    return np.array([bool(int(prob["tree"][t, node // 32]) >> (node % 32) & 1) for t in range(nodes)])


# (query heads on one key/value head, columns, tokens): 8, 16 and 32 rows, one tile of
# 128 rows and two, and one request whose rows are several units
ROWS = [(2, 64, 3), (4, 128, 4), (2, 128, 16), (3, 64, 40), (4, 128, 60), (4, 64, 150)]


@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("tree", [None, "random"])
@pytest.mark.parametrize("heads,D,T", ROWS + [(1, 128, 300)])
@pytest.mark.parametrize("ctx", [0, 50, 3000])
def test_one_value_that_is_not_finite(q, ws, ctx, heads, D, T, tree, bad):
    """fp16 rows: nodes with one infinity or NaN each, in columns of their own.
    The other columns count once, for every token, and the bad ones only for
    tokens that see them; the same on every run."""
    prob = ref.problem([ctx], [T], heads, 1, D, 16, tree=tree, seed=T, words=10 if tree else None)
    nodes = sorted({1, T // 3, T // 2, T - 1})
    clean, p = copy(prob), copy(prob)
    for column, node in enumerate(nodes):
        at = (prob["table"][0, (ctx + node) // 16], 0, (ctx + node) % 16, 7 * column)
        clean["v"][at], p["v"][at] = 0.0, bad
    want, allow = ref.attention(clean, D ** -0.5)
    first = call(q, p, ws)
    got = first.cpu().numpy().astype(np.float64)
    shown = np.zeros(got.shape, dtype=bool)
    for column, node in enumerate(nodes):
        shown[seeing(p, node, T), :, 7 * column] = True
    assert not np.isfinite(got[shown]).any()
    assert np.all(np.abs(got - want)[~shown] <= allow[~shown])
    for _ in range(10):
        again = call(q, p, ws)
        assert torch.equal(first.view(torch.int16)[torch.from_numpy(~shown).cuda()],
                           again.view(torch.int16)[torch.from_numpy(~shown).cuda()])
    assert q.qmv_device_status() == 0


def test_requests_with_such_a_value_between_others(q, ws):
    """Units with and without one in turn on the same blocks of threads."""
    R, T = 200, 80
    prob = ref.problem([(5 * r) % 60 for r in range(R)], [T] * R, 8, 4, 64, 16, seed=5)
    clean, p = copy(prob), copy(prob)
    for r in range(0, R, 3):
        j = int(prob["kv_len"][r]) - T + 1
        at = (prob["table"][r, j // 16], slice(None), j % 16, 9)
        clean["v"][at], p["v"][at] = 0.0, np.inf
    want, allow = ref.attention(clean, 0.125)
    for _ in range(5):
        got = call(q, p, ws).cpu().numpy().astype(np.float64)
        shown = np.zeros(got.shape, dtype=bool)
        for r in range(0, R, 3):
            shown[r * T + 1:(r + 1) * T, :, 9] = True
        assert not np.isfinite(got[shown]).any()
        assert np.all(np.abs(got - want)[~shown] <= allow[~shown])
    assert q.qmv_device_status() == 0


@pytest.mark.parametrize("big", [1e6, 1e10, 1e30, 2e36])
@pytest.mark.parametrize("tree", [None, "random"])
@pytest.mark.parametrize("heads,D,T", ROWS)
@pytest.mark.parametrize("ctx", [0, 50, 3000])
def test_large_value_scales_of_unseen_nodes(q, ws, ctx, heads, D, T, tree, big):
    """8-bit rows: a node whose value row has a large finite scale leaves the
    tokens that do not see it within the allowance of what they do see."""
    prob = ref.problem([ctx], [T], heads, 1, D, 16, q8=True, tree=tree, seed=T, words=5 if tree else None)
    for node in {T - 1, T // 2, 1}:
        p = copy(prob)
        at = ctx + node
        p["v_scale"][p["table"][0, at // 16], :, at % 16] = big
        off = ~seeing(p, node, T)
        assert off.any()
        want, allow = ref.attention(prob, D ** -0.5)
        got = call(q, p, ws).cpu().numpy().astype(np.float64)
        assert np.all(np.abs(got[off] - want[off]) <= allow[off]), (node, np.nanmax(np.abs(got[off] - want[off])))
    assert q.qmv_device_status() == 0


@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("heads,D,T", ROWS)
@pytest.mark.parametrize("ctx", [0, 50, 9000])
def test_a_seen_value_that_is_not_finite_shows_whatever_its_weight(q, ws, ctx, heads, D, T, bad):
    """fp16 rows: infinity or NaN times a weight too small for fp16 or fp32 is
    still not a finite number."""
    prob = ref.problem([ctx], [T], heads, 1, D, 16, seed=T)
    one = prob["q"][0, 0].copy()
    prob["q"][:] = one
    unit = one.astype(np.float64) / np.linalg.norm(one.astype(np.float64))
    far = -100.0 / (np.linalg.norm(one.astype(np.float64)) * D ** -0.5)      # a score of -100
    for low in (1, ctx + T - 1):        # node 1 alone, then all but the first place
        p = copy(prob)
        node = 1
        for j in range(ctx + T - low if low > 1 else ctx + node, ctx + T if low > 1 else ctx + node + 1):
            p["k"][p["table"][0, j // 16], 0, j % 16] = (unit * far).astype(np.float16)
        at = ctx + node
        p["v"][p["table"][0, at // 16], 0, at % 16, 5] = bad
        got = call(q, p, ws).cpu().numpy().astype(np.float64)
        on = seeing(p, node, T)
        assert not np.isfinite(got[on][:, :, 5]).any(), low
        assert np.isfinite(got[~on]).all()
    assert q.qmv_device_status() == 0
