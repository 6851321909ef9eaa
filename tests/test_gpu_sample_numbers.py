"""qmv_sample refuses a number outside its range before it runs."""
import numpy as np
import pytest

from tests.test_gpu_kv_pages import q  # noqa: F401
from tests.test_gpu_sample import check, rows
from tests.test_sample_numbers import BAD, INF, NAN

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_numbers(q):  # noqa: F811
    x, u = torch.zeros(3, 50, device="cuda"), torch.zeros(3, device="cuda")
    for kw in BAD + [dict(top_k=k) for k in (1.5, INF, -INF, NAN)] + [dict(temperature=np.float32(1e-30))]:
        with pytest.raises(ValueError):
            q.qmv_sample(x, u, **kw)
    assert q.qmv_device_status() == 0


def test_the_ends_of_the_range(q):  # noqa: F811
    x = rows("normal", 3, 700, 2)
    for T in (2.0 ** -64, 2.0 ** 64, np.float32(2.0 ** -64)):
        for kw in (dict(), dict(top_k=1 << 40), dict(top_k=np.int64(7), top_p=2.0)):
            check(q, x, [0.1, 0.5, 0.9], T=T, **kw)
    assert q.qmv_device_status() == 0
