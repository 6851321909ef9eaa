"""Queries of many short units, one after another in a block's shared memory:
each unit's products read its own."""
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


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("R,T,heads,hk,D", [(150, 20, 16, 8, 64), (60, 40, 16, 8, 128), (90, 60, 16, 4, 64)])
def test_many_short_units(q, R, T, heads, hk, D, q8):
    """1200, 480 and 360 units of 40, 80 and 240 rows over a block or two of
    places: two to eight to a block of threads; the same bits call after call."""
    prob = ref.problem([(7 * r) % 90 for r in range(R)], [T] * R, heads, hk, D, 16, q8=q8, seed=R)
    ws = q.qmv_tree_attn_workspace()
    first = call(q, prob, ws)
    for _ in range(20):
        assert torch.equal(first, call(q, prob, ws))
    check(q, prob, ws)
