"""The bounded waits of attention over the paged cache, made to run out without
a GPU fault: a copy that never arrives ends in QMV_DEV_TIMEOUT and NaN where it
was needed, other outputs are whole, and the next call is complete and clean."""
import os
import subprocess
import sys

import numpy as np
import pytest

from tests import kv_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("T,q8", [(1, False), (4, True), (40, False), (40, True)])
def test_wait_gives_up_and_recovers(tmp_path, T, q8):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import weight_quantized_decode_gb300 as q
    out = tmp_path / "y.npz"
    r = subprocess.run([sys.executable, "-m", "tests._give_up_attn_child", str(out), str(T), str(int(q8))],
                       env=dict(os.environ, QMV_TEST_SKIP_COPY="attn:1"), cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    res = np.load(out)
    prob = ref.problem([130000, 500], [T, T], 8, 2, 64, 32, q8=q8, seed=T)
    want, allow = ref.attention(prob, 0.125)
    assert int(res["s1"][0]) == q.QMV_DEV_TIMEOUT and int(res["s2"][0]) == 0
    y1, y2 = res["y1"].astype(np.float64), res["y2"].astype(np.float64)
    assert np.all(np.abs(y2 - want) <= allow)
    lost = np.isnan(y1)
    # the first key/value head (four query heads) of the first request, and nothing of the other request
    assert lost[:T, :4].any() and not lost[T:].any()
    assert np.all(np.abs(y1 - want)[~lost] <= allow[~lost])
