"""What the token kernels' sources have to keep to where no run would show it: instructions that a warp has to execute
together (.aligned) follow code in which its threads may have parted."""

import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "conv2d_implicit_gemm_gb300", "csrc")
TOKEN = [p for n in ("attn_*.cu*", "linear_*.cu*", "qk_norm_rope.cu", "token*.cuh") for p in glob.glob(os.path.join(CSRC, n))]


def lines(path):
    with open(path) as f:
        return [re.sub(r"//.*", "", s).strip() for s in f]


def test_cluster_barriers_gather_the_warp_first():
    found = 0
    for path in TOKEN:
        code = [s for s in lines(path) if s]
        for i, s in enumerate(code):
            if "barrier.cluster.arrive" in s and "aligned" in s:
                found += 1
                assert code[i - 1] == "__syncwarp();", path
    assert found


def test_named_barriers_gather_the_warp_first():
    found = 0
    for path in TOKEN:
        code = [s for s in lines(path) if s]
        for i, s in enumerate(code):
            if s.startswith("named_barrier_sync("):
                found += 1
                assert code[i - 1] == "__syncwarp();", path
    assert found


def test_tensor_memory_is_read_by_whole_warps_after_single_threads_arrived():
    """No read of tensor memory between `if (one thread) arrive` and the next point where the warp comes together."""
    together = re.compile(r"__syncwarp|__all_sync|__any_sync|__shfl|__syncthreads|cluster_sync")
    for path in TOKEN:
        parted = False
        for s in lines(path):
            if re.search(r"if \((r|lane) == 0", s):
                parted = True
            if together.search(s):
                parted = False
            if "tmem_ld" in s and "(" in s and "__device__" not in s:
                assert not parted, (path, s)
