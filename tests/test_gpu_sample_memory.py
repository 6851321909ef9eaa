"""qmv_sample where rows are read again from memory: fp16 as well as fp32, by clusters of one, two, four and eight CTAs,
in rows that begin off a 16-byte boundary."""
import numpy as np
import pytest

from tests import step_reference as ref
from tests.test_gpu_kv_pages import dev, q  # noqa: F401
from tests.test_gpu_sample import FILTERS, rows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# On 152 SMs: one CTA to a row, two, four, eight.
SIZES = [(160, 32003), (330, 70001), (64, 128256), (20, 262144)]


def padded(x, shift):
    wide = torch.full((x.shape[0], x.shape[1] + 8 + shift), float("nan"), dtype=x.dtype, device="cuda")
    wide[:, shift:shift + x.shape[1]] = x
    return wide[:, shift:shift + x.shape[1]]


@pytest.mark.parametrize("R,V", SIZES)
@pytest.mark.parametrize("kind", ["text", "ties", "masked", "normal"])
def test_fp16_rows(q, R, V, kind):  # noqa: F811
    """Every row as its fp32 copy has it, and as a few rows by themselves, which are held in shared memory; some against
    the definition."""
    x = rows(kind, R, V, R, True)
    u = np.random.RandomState(V).rand(R).astype(np.float32)
    half, ud = dev(x), dev(u)
    single = half.float()
    for i, (T, k, p, m) in enumerate(FILTERS):
        got = q.qmv_sample(padded(half, (1, 3, 7, 0)[i % 4]), ud, T, k, p, m)
        wide = q.qmv_sample(padded(single, (1, 2, 3, 0)[i % 4]), ud, T, k, p, m)
        few = q.qmv_sample(half[5:8].contiguous(), ud[5:8], T, k, p, m)
        assert torch.equal(got.token, wide.token) and torch.equal(got.prob, wide.prob)
        assert torch.equal(got.token[5:8], few.token) and torch.equal(got.prob[5:8], few.prob)
        token, prob = got.token.cpu().numpy(), got.prob.cpu().numpy()
        for r in (0, R // 2, R - 1):
            match = [(pr, a) for t, pr, a in ref.sample_choices(x[r], u[r], T, k, p, m) if t == token[r]]
            assert match and any(abs(prob[r] - pr) <= a for pr, a in match), (r, token[r])
    assert q.qmv_device_status() == 0


@pytest.mark.parametrize("R,V", SIZES)
@pytest.mark.parametrize("f16", [False, True])
def test_rows_that_are_refused_or_empty(q, R, V, f16):  # noqa: F811
    x = rows("text", R, V, 3, f16)
    x[1] = -np.inf
    x[2, V - 1], x[4, 0] = np.nan, np.inf
    x[7] = -np.inf
    x[7, V - 1] = -60000.0
    for T, k, p, m in ((1.0, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 50, 1.0, 0.0), (0.7, 700, 0.9, 0.1)):
        got = q.qmv_sample(padded(dev(x), 5), torch.full((R,), 0.5, device="cuda"), T, k, p, m)
        t, pr = got.token.tolist(), got.prob.cpu().numpy()
        assert [t[r] for r in (1, 2, 4, 7)] == [-1, -1, -1, V - 1]
        assert pr[1] == 0 and np.isnan(pr[[2, 4]]).all() and pr[7] == 1
        assert min(t[r] for r in range(R) if r not in (1, 2, 4)) >= 0
        assert q.qmv_device_status() == q.QMV_DEV_BAD_VALUE
