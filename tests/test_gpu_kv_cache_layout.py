"""Layouts of a cache's tensors that a KvCache takes and refuses."""
import pytest

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


@pytest.mark.parametrize("q8", [False, True])
def test_one_head_of_any_stride(q, q8):
    """With one key/value head a pool kept as [n_pages, page, 1, head_dim] is the
    same memory as [n_pages, 1, page, head_dim]: it is taken, and its rows are
    written and read like the other's."""
    n, page, D = 5, 16, 64
    dt = torch.int8 if q8 else torch.float16
    plain = q.qmv_kv_cache(n, 1, page, D, dt)
    k, v = (torch.zeros(n, page, 1, D, dtype=dt, device="cuda") for _ in range(2))
    scales = [torch.zeros(n, 1, page, device="cuda") for _ in range(2)] if q8 else []
    turned = q.KvCache(k.transpose(1, 2), v.transpose(1, 2), *scales)
    x = torch.randn(20, 6 * D, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    slots, table = torch.arange(30, 50, **i32), torch.tensor([[1, 2, 3]], **i32)
    start, kv_len = torch.tensor([0, 20], **i32), torch.tensor([34], **i32)
    outs = []
    for c in (plain, turned):
        qo = q.qmv_kv_append(x, c, slots, 4)
        outs.append(q.qmv_tree_attn(qo, c, table, start, kv_len))
    assert torch.equal(plain.k, turned.k) and torch.equal(plain.v, turned.v) and plain.k.any()
    assert torch.equal(*outs) and outs[0].any()
    assert q.qmv_device_status() == 0


def test_rows_that_are_not_dense_are_refused(q):
    for t in (torch.zeros(4, 16, 2, 64, device="cuda").half().transpose(1, 2),       # two heads, by place
              torch.zeros(4, 1, 32, 64, device="cuda").half()[:, :, ::2],            # every second row
              torch.zeros(4, 1, 16, 128, device="cuda").half()[..., ::2]):           # every second column
        with pytest.raises(ValueError):
            q.KvCache(t, t)
