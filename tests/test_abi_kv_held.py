"""Host validation of qmv_kv_pages_held: its two arrays may be missing, and
have to be aligned (nothing runs on a GPU here)."""
import pytest

from tests.test_abi_kv import FAKE, PAGES, _call, lib  # noqa: F401

HELD = {}
for name, value in PAGES.items():
    HELD[name] = value
    if name == "table":
        HELD["held"] = FAKE
    if name == "head_out":
        HELD["held_out"] = FAKE


@pytest.mark.parametrize("kw,code", [
    (dict(held=FAKE + 2), 2), (dict(held_out=FAKE + 1), 2), (dict(held=None, held_out=None, len=None), 1),
    (dict(start=None), 1), (dict(page=24), 3), (dict(T=-1), 3),
    (dict(R=0, T=0, start=None, head_out=None, held=None, held_out=None), 0),
])
def test_pages_held(lib, kw, code):  # noqa: F811
    assert _call(lib.qmv_kv_pages_held, HELD, **kw) == code
