"""qmv_sample's settings as one number for all rows: checked on the host as the fp32 numbers that the kernel takes."""
import ctypes

import pytest

import weight_quantized_decode_gb300 as q
from tests.test_abi_kv import _call, lib  # noqa: F401
from tests.test_abi_step import SAMPLE

NAN, INF = float("nan"), float("inf")
LOW, HIGH = 2.0 ** -64, 2.0 ** 64
BAD = [dict(temperature=v) for v in (-1.0, 1e-50, 1e-30, LOW * (1 - 2.0 ** -23), 2 * HIGH, 1e24, 1e300, INF, NAN, 10 ** 400)] + \
      [dict(top_p=v) for v in (-0.5, -1e-50, NAN, -INF)] + [dict(min_p=v) for v in (-0.1, 1.5, INF, NAN)]
GOOD = [dict(temperature=v) for v in (0, 0.0, -0.0, 1, LOW, HIGH)] + [dict(top_p=v) for v in (0, 1e-50, 1, 2.0, INF)] + \
       [dict(min_p=v) for v in (0, 1e-50, 1)]


def settings(temperature=1.0, top_p=1.0, min_p=0.0):
    return temperature, top_p, min_p


@pytest.mark.parametrize("kw", BAD)
def test_numbers_that_are_refused(kw):
    with pytest.raises(ValueError):
        q._sample_numbers("qmv_sample", *settings(**kw), 0)


@pytest.mark.parametrize("k", [1.5, INF, -INF, NAN])
def test_top_k_is_a_whole_number(k):
    with pytest.raises(ValueError):
        q._sample_numbers("qmv_sample", *settings(), k)


@pytest.mark.parametrize("kw", GOOD)
@pytest.mark.parametrize("k", [0, -3, 50.0, 1 << 70])
def test_numbers_that_are_taken(kw, k):
    alike, top_k = q._sample_numbers("qmv_sample", *settings(**kw), k)
    assert list(alike) == list((ctypes.c_float * 3)(*settings(**kw)))
    assert top_k == max(-1, min(int(k), 1 << 19))


@pytest.mark.parametrize("kw", [kw for kw in BAD if kw != dict(temperature=10 ** 400) and 1e-50 not in kw.values()
                                and -1e-50 not in kw.values()])
@pytest.mark.parametrize("R", [0, 2])
def test_the_c_entry(lib, kw, R):  # noqa: F811
    alike = (ctypes.c_float * 3)(*settings(**kw))
    assert _call(lib.qmv_sample, SAMPLE, all=alike, R=R) == 3


@pytest.mark.parametrize("kw", GOOD)
def test_the_c_entry_takes(lib, kw):  # noqa: F811
    """(No rows: nothing runs.)  And numbers that an array stands in for do not count."""
    assert _call(lib.qmv_sample, SAMPLE, all=(ctypes.c_float * 3)(*settings(**kw)), R=0) == 0
    for i, name in enumerate(("temperature", "top_p", "min_p")):
        numbers = list(settings())
        numbers[i] = NAN
        assert _call(lib.qmv_sample, SAMPLE, all=(ctypes.c_float * 3)(*numbers), R=0, **{name: 1 << 20}) == 0
