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
