"""What the norms around a branch take beside the plain call, over few rows, many rows (teams with a ring) and long rows:
kinds, gates and absent parts against the definitions in 64 bits, with the tolerances of tests/test_gpu_block.py."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from tests.test_gpu_block import check_block


# a part of a warp (8 and 16 lanes), one warp, several, of whole pieces and of single values; a CTA a row; long rows
WIDTHS = [72, 77, 200, 333, 1001, 1536, 4096, 5000, 16000, 17000]


@pytest.mark.parametrize("kind,total_kind", [("fp16", "fp16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("t", [5, 700])
@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("post,pre", [("none", "rms"), ("layer", "none"), ("none", "none")])
def test_a_norm_of_no_kind_takes_no_weight_or_bias(t, n, post, pre, kind, total_kind):
    check_block(t, n, kind, total_kind, post=post, pre=pre, per=max(1, t // 3), seed=n)
