"""The paged-cache calls on a stream that is not the current one: whose memory
their temporary and their outputs are."""
import numpy as np
import pytest

from tests import kv_reference as ref
from tests.test_gpu_tree_attn import dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

WORKSPACE = 18      # its place among the library call's arguments


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import weight_quantized_decode_gb300 as m
    m.lib()
    m.qmv_device_status()
    yield m
    torch.cuda.synchronize()


def attn_args(q, prob):
    c = q.KvCache(*(dev(prob[n]) for n in ("k", "v", "k_scale", "v_scale")))
    return dev(prob["q"]), c, dev(prob["table"]), dev(prob["start"]), dev(prob["kv_len"])


def handles(s):
    return s, s.cuda_stream      # a torch stream, and the plain handle


@pytest.mark.parametrize("which", [0, 1])
def test_a_temporary_workspace_stays_with_its_stream(q, which, monkeypatch):
    """After a call on another stream without a workspace, the current stream's
    next allocation is not the memory that the call's kernels still use.  (The
    launch itself is left out, so that nothing runs in that memory here.)"""
    args = attn_args(q, ref.problem([700], [3], 8, 2, 64, 16, seed=8))
    n = q.lib().qmv_tree_attn_workspace()
    s = torch.cuda.Stream()
    seen = []
    monkeypatch.setattr(q, "_call_on", lambda fn, index, stream, a: seen.append(a[WORKSPACE]))
    q.qmv_tree_attn(*args, stream=handles(s)[which])
    other = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert abs(other.data_ptr() - seen[0]) >= n


def test_calls_without_a_workspace_on_two_streams(q):
    """Two streams' calls, each with the workspace made for it, between
    allocations of the same size on the current stream."""
    probs = [ref.problem([9000], [8], 8, 2, 128, 32, seed=1), ref.problem([5000], [90], 8, 2, 128, 32, seed=2)]
    args = [attn_args(q, p) for p in probs]
    alone = [q.qmv_tree_attn(*a) for a in args]
    n = q.lib().qmv_tree_attn_workspace()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(12):
        got.append([q.qmv_tree_attn(*a, stream=handles(s)[i % 2]) for a, s in zip(args, streams)])
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(alone, pair):
            assert torch.equal(a, b)
    assert q.qmv_device_status() == 0


@pytest.mark.parametrize("which", [0, 1])
def test_outputs_are_not_memory_the_current_stream_gave_up(q, which, monkeypatch):
    """A call on another stream does not write its output where work of the
    current stream, whose tensor is gone, may still be running."""
    prob = ref.problem([60, 9], [40, 30], 8, 2, 128, 16, seed=8)
    args = attn_args(q, prob)
    ws = q.qmv_tree_attn_workspace()
    R, T, i32 = 2, 70, dict(dtype=torch.int32, device="cuda")
    lens, free, table = torch.zeros(R, **i32), torch.arange(9, **i32), torch.full((R, 4), -1, **i32)
    qkv, slots = torch.zeros(T, (8 + 4) * 128, device="cuda"), torch.arange(T, **i32)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    monkeypatch.setattr(q, "_call_on", lambda fn, index, stream, a: None)      # nothing is launched
    for call, shape, dtype in (
            (lambda **kw: q.qmv_tree_attn(*args, workspace=ws, **kw), (T, 8, 128), torch.float16),
            (lambda **kw: q.qmv_kv_append(qkv, args[1], slots, 8, **kw), (T, 8, 128), torch.float16),
            (lambda **kw: q.qmv_kv_pages(lens, lens, free, table, 16, T, **kw).start, (2 * R + 2 + 3 * T,), torch.int32)):
        gone = torch.empty(shape, dtype=dtype, device="cuda")
        lo, n = gone.data_ptr(), gone.nbytes
        del gone
        out = call(stream=handles(s)[which])
        assert abs(out.data_ptr() - lo) >= n
        kept = call()                                  # on the current stream its own memory will do
        assert kept.data_ptr() == lo and kept.shape == out.shape and kept.dtype == out.dtype


def test_outputs_of_another_stream_in_a_graph(q):
    """Calls that name the capturing stream, and calls that name one forked from it."""
    args = attn_args(q, ref.problem([900, 30], [8, 3], 8, 2, 64, 16, seed=3))
    ws = q.qmv_tree_attn_workspace()
    want = q.qmv_tree_attn(*args, workspace=ws)
    torch.cuda.synchronize()
    s, fork = torch.cuda.Stream(), torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            a = q.qmv_tree_attn(*args, workspace=ws, stream=s)
            fork.wait_stream(s)
            b = q.qmv_tree_attn(*args, workspace=ws, stream=fork)
            s.wait_stream(fork)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)
    assert q.qmv_device_status() == 0
