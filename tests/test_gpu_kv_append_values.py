"""8-bit cache rows with values that are not finite: the row says so."""
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


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
def test_a_row_that_is_not_finite(q, D, dtype, bad):
    """One value of a key row and one of another token's value row: their scales
    are not finite, the other rows as before; a token that sees the row is NaN."""
    c, clean = (q.qmv_kv_cache(4, 2, 16, D, torch.int8) for _ in range(2))
    x = torch.randn(5, 6 * D, device="cuda").to(dtype)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    q.qmv_kv_append(x, clean, i32(0, 1, 2, 3, 4), 2)
    y = x.clone()
    y[1, 2 * D + 7] = bad              # token 1's key row of head 0
    y[3, 5 * D + 1] = bad              # token 3's value row of head 1
    qo = q.qmv_kv_append(y, c, i32(0, 1, 2, 3, 4), 2)
    want = torch.ones(2, 5, dtype=torch.bool, device="cuda")
    k_ok, v_ok = want.clone(), want.clone()
    k_ok[0, 1] = v_ok[1, 3] = False
    for ok, name in ((k_ok, "k"), (v_ok, "v")):
        got, same = getattr(c, name + "_scale")[0, :, :5], getattr(clean, name + "_scale")[0, :, :5]
        assert torch.equal(torch.isfinite(got), ok) and torch.equal(got[ok], same[ok])
        assert torch.equal(getattr(c, name)[0, :, :5][ok], getattr(clean, name)[0, :, :5][ok])
    out = q.qmv_tree_attn(qo, c, i32(0).view(1, 1), i32(0, 5), i32(5))
    seen = torch.isfinite(out).all(-1)                             # [token, head]: a chain
    assert seen.tolist() == [[True, True], [False, True], [False, True], [False, False], [False, False]]
    assert q.qmv_device_status() == 0
