"""rotary_axes with sections that can be read only once."""
import numpy as np
import pytest

import weight_quantized_decode_gb300 as q


@pytest.mark.parametrize("sections", [(4, 2, 2), (16, 24, 24), (5,), (0, 3), (2, 0, 7, 1)])
@pytest.mark.parametrize("turns", [False, True])
def test_an_iterator(sections, turns):
    want = q.rotary_axes(sections, turns)
    assert len(want) == sum(sections)
    assert q.rotary_axes((s for s in sections), turns) == want
    assert q.rotary_axes(np.array(sections), turns) == want
