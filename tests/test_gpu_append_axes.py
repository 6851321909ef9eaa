"""qmv_kv_append gives the same rows whatever holds the axes."""
import numpy as np
import pytest

import weight_quantized_decode_gb300 as m
from tests.test_gpu_kv_pages import dev, q  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_holders_of_axes(q):  # noqa: F811
    rs = np.random.RandomState(1)
    T, H, hk, D = 5, 4, 2, 64
    axes = m.rotary_axes((12, 10, 10), turns=True)
    cache = q.qmv_kv_cache(1, hk, 16, D)
    angle = rs.rand(40, D // 2)
    call = dict(pos=dev(rs.randint(0, 40, (3, T)).astype(np.int32)), cos=dev(np.cos(angle).astype(np.float32)),
                sin=dev(np.sin(angle).astype(np.float32)))
    qkv, slots = dev(rs.randn(T, (H + 2 * hk) * D).astype(np.float32)), dev(np.arange(T, dtype=np.int32))
    want = q.qmv_kv_append(qkv, cache, slots, H, axes=axes, **call)
    for t in ("int8", "int32", "int64"):
        got = q.qmv_kv_append(qkv, cache, slots, H, axes=np.array(list(axes), dtype=t), **call)
        assert torch.equal(got, want)
    for bad in (32, np.array([0, 1, 2, 0, 1, 2, 0, 1], dtype=np.int32), [0] * 31 + [3], [0] * 33):
        with pytest.raises((TypeError, ValueError)):
            q.qmv_kv_append(qkv, cache, slots, H, axes=bad, **call)
    assert q.qmv_device_status() == 0
