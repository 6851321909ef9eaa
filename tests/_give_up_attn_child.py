"""Child process for test_gpu_give_up_attn: QMV_TEST_SKIP_COPY="attn:1" (read
once per process) makes the first attention launch skip a copy whose bytes a
barrier expects.  Runs the call, reads the status word, then repeats it and
reads the status again.
Usage: python -m tests._give_up_attn_child OUT.npz T q8(0|1)"""
import sys

import numpy as np
import torch

import weight_quantized_decode_gb300 as q
from tests import kv_reference as ref
from tests.test_gpu_tree_attn import call


def main():
    out, T, q8 = sys.argv[1], int(sys.argv[2]), sys.argv[3] == "1"
    prob = ref.problem([130000, 500], [T, T], 8, 2, 64, 32, q8=q8, seed=T)
    ws = q.qmv_tree_attn_workspace()
    got = []
    for _ in range(2):
        y = call(q, prob, ws)
        torch.cuda.synchronize()
        got += [y.float().cpu().numpy(), np.array([q.qmv_device_status()])]
    np.savez(out, y1=got[0], s1=got[1], y2=got[2], s2=got[3])


if __name__ == "__main__":
    main()
