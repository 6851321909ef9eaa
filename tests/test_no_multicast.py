"""The library is the same on one GPU and on several, where copies with cluster multicast are not used: it has none."""
import glob
import os

import weight_quantized_decode_gb300 as q


def test_no_multicast_copy():
    csrc = os.path.join(os.path.dirname(q.__file__), "csrc")
    files = [f for f in sorted(glob.glob(os.path.join(csrc, "*"))) if f.endswith((".cu", ".cuh", ".h"))]
    assert len(files) > 20
    for f in files:
        assert "multicast::cluster" not in open(f, encoding="utf-8").read(), os.path.basename(f)
