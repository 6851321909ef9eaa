"""A request without a next token (nothing new in the step, or nothing left to draw) goes through the next step, and
leaves the others as they are."""
import numpy as np
import pytest

from tests.test_gpu_decode_drafts import VOCAB, decoder, ints
from tests.test_gpu_kv_pages import dev, q  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

PARENTS = [-1, 0, 0, 2]


@pytest.mark.parametrize("why", ["idle", "masked"])
def test_next_is_none(q, why):  # noqa: F811
    from weight_quantized_decode_gb300 import decode_block as b
    rs = np.random.RandomState(4)
    prompt, mask = dev(rs.randint(0, VOCAB, 30).astype(np.int32)), b.tree_mask(PARENTS)
    drafts = rs.randint(0, VOCAB, 3).tolist()
    rows = {}
    for stand_in in (-1, 0):            # the token as it comes, and the one that it is looked up as
        d = decoder(2)
        d.logits(prompt, ints(20, 10))
        n, T = ((4, 0), 4) if why == "idle" else ((4, 4), 8)
        tree = dev(np.concatenate([mask] * (T // 4)))
        logits, maps = d.logits(ints(*([7] + drafts) * (T // 4)), ints(*n), tree)
        if why == "masked":
            logits[4:] = -float("inf")
        drawn = q.qmv_sample(logits, torch.full((T,), 0.5, device="cuda"), 0.0)
        got = d.block.accept(ints(*([7] + drafts) * (T // 4)), drawn.token, maps, tree)
        assert int(got.next[0]) >= 0 and int(got.next[1]) == -1
        first = got.next.clone() if stand_in < 0 else got.next.clamp(min=0)
        tokens = torch.cat([first[:1], ints(*drafts), first[1:], ints(*drafts)])
        out = d.verify(tokens, ints(4, 4), torch.full((8,), 0.5, device="cuda"), dev(np.concatenate([mask] * 2)),
                       temperature=0.0)
        assert (out.next >= 0).all()
        # and one that gets nothing more, beside the padding that its places are
        later, _ = d.logits(torch.cat([out.next[:1], ints(-1, -1)]), ints(1, 0))
        rows[stand_in] = later[0]
        assert torch.isfinite(later[0]).all()
    assert torch.equal(rows[-1], rows[0])
    assert q.qmv_device_status() == 0
