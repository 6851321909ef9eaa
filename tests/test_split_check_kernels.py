"""Host-only check of the split of work over CTAs with the sizes and costs that
the attention kernels are compiled with (no GPU)."""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "weight_quantized_decode_gb300", "csrc")


def test_every_block_is_taken_once(tmp_path):
    nvcc = next((c for c in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc") if c and os.path.exists(c)), None)
    if nvcc is None:
        pytest.skip("nvcc not found")
    exe = str(tmp_path / "split_check_kernels")
    r = subprocess.run([nvcc, "-std=c++17", "-O2", "--expt-relaxed-constexpr", "-gencode",
                        "arch=compute_103a,code=sm_103a", "-o", exe,
                        os.path.join(HERE, "plan_check", "split_check_kernels.cu")],
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:]
    assert " 0 failures" in r.stdout, r.stdout


def test_the_kernels_have_no_sizes_of_their_own():
    """Both kernels take their split from where the check takes it."""
    for name, split in (("rows", "RowsSplit"), ("tiles", "TilesSplit")):
        with open(os.path.join(CSRC, f"qmv_attn_{name}.cu")) as f:
            source = f.read()
        for what in ("kBlock", "kCost"):
            assert re.findall(rf"constexpr int {what} = (.*);", source) == [f"{split}::{what}"], (name, what)
