"""What the norms around a branch take beside the plain call, over few rows, many rows (teams with a ring) and long rows:
kinds, gates and absent parts against the definitions in 64 bits, with the tolerances of tests/test_gpu_block.py."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from tests._tokens import block_norm, done, strided
from tests.test_gpu_block import check_block


# a part of a warp (8 and 16 lanes), one warp, several, of whole pieces and of single values; a CTA a row; long rows
WIDTHS = [72, 77, 200, 333, 1001, 1536, 4096, 5000, 16000, 17000]


@pytest.mark.parametrize("kind,total_kind", [("fp16", "fp16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("t", [5, 700])
@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("post,pre", [("none", "rms"), ("layer", "none"), ("none", "none")])
def test_a_norm_of_no_kind_takes_no_weight_or_bias(t, n, post, pre, kind, total_kind):
    check_block(t, n, kind, total_kind, post=post, pre=pre, per=max(1, t // 3), seed=n)


# ---------------------------------------------------------------- many rows of every form
MANY = [(72, 0, 0), (96, 8, 8), (200, 0, 0), (333, 0, 0), (500, 3, 1), (1001, 0, 0), (1536, 0, 0), (2048, 8, 4), (4096, 0, 0),
        (5000, 0, 0), (8000, 0, 0)]


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("n,pad,shift_at", MANY)
def test_many_rows_of_each_kind(n, pad, shift_at, post, pre):
    check_block(700, n, "bf16", "fp32", post=post, pre=pre, per=200, alpha=0.7, beta=-1.3, pad=pad, shift_at=shift_at, seed=n)


@pytest.mark.parametrize("gate", ["none", "channel", "groups"])
@pytest.mark.parametrize("gate_act", ["plain", "tanh", "sigmoid"])
@pytest.mark.parametrize("n,pad,shift_at", MANY)
def test_many_rows_with_each_gate(n, pad, shift_at, gate, gate_act):
    check_block(700, n, "fp16", gate=gate, gate_act=gate_act, per=150, alpha=-0.3, beta=2.1, pad=pad, shift_at=shift_at, seed=n)


@pytest.mark.parametrize("without", ["scale", "shift", "bias", "weight", "residual", "total", "y"])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("n,pad,shift_at", MANY)
def test_many_rows_without_a_part(n, pad, shift_at, kind, without):
    check_block(700, n, kind, **{without: False}, pre="layer", gate_act="sigmoid", per=230, pad=pad, shift_at=shift_at, seed=n)


@pytest.mark.parametrize("n,pad,shift_at", MANY)
def test_many_rows_with_nothing_beside_them(n, pad, shift_at):
    check_block(700, n, "fp16", "fp32", gate="none", scale=False, shift=False, bias=False, weight=False, residual=False, pad=pad,
                shift_at=shift_at, seed=n)


@pytest.mark.parametrize("per", [1, 2, 699])
@pytest.mark.parametrize("n", [96, 333, 2048])
def test_many_rows_of_groups_of_any_size(n, per):
    check_block(700, n, "bf16", gate_act="tanh", per=per, seed=n)


@pytest.mark.parametrize("n", [96, 333, 2048, 5000])
def test_many_rows_with_padding_among_them(n):
    groups = np.random.default_rng(n).integers(-1, 5, 700)
    groups[[0, 1, 350, 699]] = -1, 2 ** 31 - 1, -2 ** 31, 4
    check_block(700, n, "fp16", count=4, groups=groups, inplace=True)


@pytest.mark.parametrize("n,pad,shift_at", MANY)
def test_many_rows_far_from_zero(n, pad, shift_at):
    """A mean 500 times the deviation: off by what the mean's own rounding is, relative to the deviation."""
    check_block(700, n, "fp32", post="layer", pre="layer", mean=1000.0, gate="none", scale=False, shift=False, pad=pad,
                shift_at=shift_at)


@pytest.mark.parametrize("n", [96, 333, 1001, 2048, 5000])
def test_infinities_and_nan_of_many_rows_stay_in_theirs(n):
    """Rows of NaN and of infinities, and padding rows of NaN, change nothing of the others."""
    t = 700
    x, r = strided((t, n), "bf16", 1), strided((t, n), "bf16", 2)
    groups = torch.zeros(t, dtype=torch.int32, device="cuda")
    groups[100::50] = -1
    bad = {7: float("nan"), 8: float("inf"), 333: float("-inf"), 699: float("nan")}

    def call():
        s, y = torch.zeros_like(x), torch.zeros_like(x)
        block_norm(x, r, s, y, "none", None, None, "layer", None, None, 1e-6, None, "plain", None, None, groups, 1, 1, 1.0, 1.0,
                   "bf16", "bf16")
        done()
        return s, y

    plain = call()
    for row, value in bad.items():
        x[row, row % n] = value
    x[100::50] = float("nan")
    rest = [i for i in range(t) if i not in bad]
    for got, ref in zip(call(), plain):
        assert torch.equal(got[rest], ref[rest])
        for row in bad:
            assert not got[row, row % n].isfinite()
    assert call()[1][list(bad)].isnan().all()
