"""What the Python entry points of a conditioned block's operators take where the C functions take NULL: no kernel runs here."""

import pytest

from tests.test_block_refusals import _axes


@pytest.fixture(scope="module")
def ox():
    import conv2d_implicit_gemm_gb300 as m
    return m


def test_no_pairs_need_no_axes(ox):
    _axes(ox, rot=0, pair_axes=None, t=0)
    _axes(ox, rot=0, pair_axes=b"", t=0)
    assert ox.oidnx_last_error() == ""


def test_pairs_need_their_axes(ox):
    with pytest.raises(ValueError, match="0 of 32"):
        _axes(ox, pair_axes=None)
