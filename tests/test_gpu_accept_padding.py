"""qmv_tree_accept where offsets fall: the places of sound requests are theirs, only what no request has is padding."""
import numpy as np
import pytest

from tests import step_reference as ref
from tests.test_gpu_kv_pages import dev, q  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("start", [
    [0, 5, 2, 2],              # the last one is empty and lies in front of the first one's end
    [5, 8, 0, 2],              # the last one lies in front of the first one
    [0, 40, 90, 60],           # the last one falls
    [0, 50, 10, 10, 10],
    [0, 3, 60, 1 << 30, 60],   # offsets past the end in between
    [70] * 40 + [90] + [2] * 30,
    [0, 3, 7, 20],             # nothing falls: as before
])
def test_falling_offsets(q, start):  # noqa: F811
    T, R = 100, len(start) - 1
    tokens = sampled = np.zeros(T, dtype=np.int32)
    kv_len = np.full(R, 200, dtype=np.int32)
    sound = [0 <= a <= b <= T for a, b in zip(start, start[1:])]
    end = max(b for b, s in zip(start[1:], sound) if s)
    got = q.qmv_tree_accept(dev(tokens), dev(sampled), dev(np.array(start, dtype=np.int32)), dev(kv_len))
    path = got.path.tolist()
    for r in range(R):
        a, b = start[r], start[r + 1]
        if sound[r]:            # a chain of which every node is drawn
            assert path[a:b] == list(range(b - a)), r
            assert (got.count[r], got.lens[r], got.next[r]) == (b - a, 200, 0 if b > a else -1)
        else:
            assert (got.count[r], got.lens[r], got.next[r]) == (0, 200, -1)
    if start[-1] <= T:
        assert path[end:] == [-1] * (T - end)
    assert q.qmv_device_status() == (0 if all(sound) else q.QMV_DEV_BAD_LENGTH)


def test_padding_behind_many_requests(q):  # noqa: F811
    rs = np.random.RandomState(1)
    nodes = rs.randint(0, 7, 3001)
    start = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    T = int(start[-1]) + 5000
    p = {"tokens": rs.randint(0, 2, T).astype(np.int32), "sampled": rs.randint(0, 2, T).astype(np.int32), "start": start,
         "kv_len": (nodes + 9).astype(np.int32)}
    got = q.qmv_tree_accept(*(dev(p[n]) for n in ("tokens", "sampled", "start", "kv_len")))
    assert {n: getattr(got, n).tolist() for n in got._fields} == ref.accept(**p)
    assert q.qmv_device_status() == 0
