"""Host validation of the paged-cache calls: bad arguments are refused before
any CUDA call (nothing runs on a GPU here)."""
import ctypes
import os

import pytest

import weight_quantized_decode_gb300 as q

FAKE = 1 << 20      # a 16-byte-aligned non-null address; never dereferenced here


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(q.LIB_PATH):
        from weight_quantized_decode_gb300 import build
        build.build()
    return q.lib()


def _call(f, args, **kw):
    a = dict(args)
    a.update(kw)
    return f(*a.values())


PAGES = dict(len=FAKE, n_new=FAKE, free=FAKE, n_free=4, head=FAKE, tree=None, words=0, table=FAKE, start=FAKE,
             kv_len=FAKE, slots=FAKE, pos=FAKE, request=FAKE, head_out=FAKE, R=2, width=3, page=16, n_pages=9, T=5,
             stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(len=None), 1), (dict(n_new=None), 1), (dict(free=None), 1), (dict(table=None), 1), (dict(start=None), 1),
    (dict(kv_len=None), 1), (dict(slots=None), 1), (dict(pos=None), 1), (dict(request=None), 1),
    (dict(len=FAKE + 2), 2), (dict(head=FAKE + 1), 2), (dict(tree=FAKE + 2, words=1), 2), (dict(head_out=FAKE + 2), 2),
    (dict(page=8), 3), (dict(page=24), 3), (dict(page=512), 3), (dict(R=-1), 3), (dict(T=-1), 3), (dict(T=1 << 31), 3),
    (dict(width=-1), 3), (dict(n_pages=0), 3), (dict(n_pages=1 << 28), 3), (dict(tree=FAKE, words=0), 3),
    (dict(n_free=-1), 3), (dict(R=0, T=0, start=None, head_out=None), 0),
])
def test_pages(lib, kw, code):
    assert _call(lib.qmv_kv_pages, PAGES, **kw) == code


APPEND = dict(qkv=FAKE, stride=512, f32=1, slots=FAKE, pos=FAKE, cos=FAKE, sin=FAKE, n_pos=10, rot=64, inter=0, q=FAKE,
              k=FAKE, v=FAKE, ks=None, vs=None, kind=0, T=3, Hq=4, Hkv=2, D=64, n_pages=9, page=16, page_stride=2048,
              stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(qkv=None), 1), (dict(slots=None), 1), (dict(pos=None), 1), (dict(cos=None), 1), (dict(sin=None), 1),
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(kind=1), 1), (dict(kind=1, ks=FAKE), 1),
    (dict(qkv=FAKE + 8), 2), (dict(qkv=FAKE + 4, f32=0), 2), (dict(stride=514), 2), (dict(k=FAKE + 8), 2),
    (dict(cos=FAKE + 8), 2), (dict(page_stride=2052), 2), (dict(D=96, stride=4096, page_stride=4096), 3),
    (dict(page=20), 3), (dict(Hkv=0), 3), (dict(kind=2), 3), (dict(page_stride=2040), 3), (dict(rot=72), 3),
    (dict(rot=12), 3), (dict(rot=-8), 3), (dict(stride=511), 3), (dict(T=-1), 3), (dict(n_pages=0), 3),
    (dict(n_pages=1 << 28), 3), (dict(T=0, qkv=None, slots=None), 0),
])
def test_append(lib, kw, code):
    assert _call(lib.qmv_kv_append, APPEND, **kw) == code


ATTN = dict(q=FAKE, q_stride=256, k=FAKE, v=FAKE, ks=None, vs=None, kind=0, n_pages=9, page=16, page_stride=2048,
            table=FAKE, width=3, start=FAKE, kv_len=FAKE, tree=None, words=0, scale=None, out=FAKE, ws=FAKE,
            ws_bytes=1 << 40, R=2, T=5, Hq=4, Hkv=2, D=64, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(table=None), 1), (dict(start=None), 1),
    (dict(kv_len=None), 1), (dict(out=None), 1), (dict(kind=1), 1), (dict(q=FAKE + 8), 2), (dict(q_stride=260), 2),
    (dict(k=FAKE + 8), 2), (dict(out=FAKE + 8), 2), (dict(ws=FAKE + 8), 2), (dict(tree=FAKE + 1, words=1), 2),
    (dict(D=80, q_stride=4096, page_stride=4096), 3), (dict(page=512), 3), (dict(Hq=5, q_stride=4096), 3),
    (dict(Hq=0), 3), (dict(Hkv=0), 3), (dict(q_stride=248), 3), (dict(T=-1), 3), (dict(T=1 << 25), 3), (dict(R=-1), 3),
    (dict(R=(1 << 20) + 1), 3), (dict(width=-1), 3), (dict(tree=FAKE), 3), (dict(kind=7), 3),
    (dict(scale=ctypes.byref(ctypes.c_float(float("inf")))), 3), (dict(T=0, q=None), 0), (dict(R=0, q=None), 0),
])
def test_attn(lib, kw, code):
    assert _call(lib.qmv_tree_attn, ATTN, **kw) == code


def test_no_cpu_path():
    torch = pytest.importorskip("torch")
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        q.qmv_kv_pages(i, i, i, i.view(2, 1), 16, 2)
    with pytest.raises(TypeError):
        q.KvCache(torch.zeros(2, 1, 16, 64).half(), torch.zeros(2, 1, 16, 64).half())
