"""The axes of a rotation's pairs, as qmv_kv_append takes them: whole numbers one by one, whatever holds them."""
import array

import numpy as np
import pytest

import weight_quantized_decode_gb300 as q

AXES = [0, 1, 2, 0, 1, 2, 0, 0, 3, 3, 3, 3, 1, 1, 1, 1]


@pytest.mark.parametrize("axes", [AXES, tuple(AXES), bytes(AXES), bytearray(AXES), range(4), array.array("i", AXES),
                                  *(np.array(AXES, dtype=t) for t in ("int8", "uint8", "int32", "int64", "bool")),
                                  np.array(AXES * 2, dtype="int64")[::2], memoryview(np.array(AXES, dtype="int32"))],
                         ids=lambda a: type(a).__name__ + str(getattr(a, "dtype", "")))
def test_whole_numbers(axes):
    got = q._axis_bytes("qmv_kv_append", axes)
    assert type(got) is bytes and list(got) == [int(a) for a in axes]


def test_tensors():
    torch = pytest.importorskip("torch")
    for dtype in (torch.int8, torch.int32, torch.int64, torch.uint8):
        assert list(q._axis_bytes("qmv_kv_append", torch.tensor(AXES, dtype=dtype))) == AXES
    for bad in (torch.tensor(3), torch.tensor([0.0, 1.0]), torch.tensor([[0, 1], [1, 0]])):
        with pytest.raises((TypeError, ValueError)):
            q._axis_bytes("qmv_kv_append", bad)


@pytest.mark.parametrize("axes", [32, 0, np.int64(4), True, 1.5, [0.0, 1.0], np.zeros(4), [[0, 1], [1, 0]],
                                  np.zeros((2, 2), dtype="int32"), "0012", [0, None], [0, -1], [0, 256],
                                  np.array([0, -1], dtype="int8"), np.array([0, 257], dtype="int64")], ids=str)
def test_refused(axes):
    with pytest.raises((TypeError, ValueError)):
        q._axis_bytes("qmv_kv_append", axes)
