"""Host validation of qmv_tree_accept_slots: bad arguments are refused before any CUDA call (nothing runs on a GPU
here)."""
import pytest

from tests.test_abi_kv import FAKE, _call, lib  # noqa: F401
from tests.test_abi_step import ACCEPT

WITH = {}
for _n, _v in ACCEPT.items():          # slots stand behind the tree's words
    WITH[_n] = _v
    if _n == "words":
        WITH["slots"] = FAKE


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=None), 1), (dict(sampled=None), 1), (dict(start=None), 1), (dict(kv_len=None), 1), (dict(path=None), 1),
    (dict(count=None), 1), (dict(next=None), 1), (dict(lens=None), 1), (dict(tokens=FAKE + 2), 2), (dict(tree=FAKE + 1), 2),
    (dict(slots=FAKE + 2), 2), (dict(words=0), 3), (dict(words=65537), 3), (dict(R=-1), 3), (dict(T=-1), 3),
    (dict(T=1 << 31), 3), (dict(R=1 << 31), 3), (dict(R=0, T=0, tokens=None, slots=None), 0),
])
def test_accept_slots(lib, kw, code):  # noqa: F811
    assert _call(lib.qmv_tree_accept_slots, WITH, **kw) == code
