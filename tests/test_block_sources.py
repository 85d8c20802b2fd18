"""What the sources of a conditioned block's operators have to keep to where no run would show it: instructions that a
warp has to execute together (.aligned) follow code in which its threads may have parted."""

import glob
import os
import re

from tests.test_token_sources import CSRC, lines

BLOCK = [p for n in ("cross_*.cu", "block_norm.cu", "heads_copy.cu") for p in glob.glob(os.path.join(CSRC, n))]


def test_named_barriers_gather_the_warp_first():
    found = 0
    for path in BLOCK:
        code = [s for s in lines(path) if s]
        for i, s in enumerate(code):
            if "named_barrier_sync(" in s:
                found += 1
                assert code[i - 1] == "__syncwarp();", path
    assert found


def test_tensor_memory_is_read_by_whole_warps_after_single_threads_arrived():
    """No read of tensor memory between `if (one thread) ..` and the next point where the warp comes together."""
    together = re.compile(r"__syncwarp|__all_sync|__any_sync|__shfl|__syncthreads|cluster_sync|mbar_arrive_if")
    for path in BLOCK:
        parted = False
        for s in lines(path):
            if re.search(r"if \((r|lane|tid) == 0", s):
                parted = True
            if together.search(s):
                parted = False
            if "tmem_ld" in s and "(" in s:
                assert not parted, (path, s)


def test_waits_are_bounded():
    """Every wait on a barrier in shared memory goes through the helpers that give up."""
    for path in BLOCK:
        for s in lines(path):
            assert "mbar_try_wait" not in s, path


def test_parts_of_a_row_are_measured_in_one_place():
    """The workspace's size and both kernels' strides come from cross_part_floats."""
    uses = {name: sum("cross_part_floats(" in s for s in lines(os.path.join(CSRC, name))) for name in ("block_host.cpp", "cross_token.cu")}
    assert uses == {"block_host.cpp": 1, "cross_token.cu": 2}
    for name in uses:
        assert not any(re.search(r"\bd \+ \d", s) for s in lines(os.path.join(CSRC, name))), name
