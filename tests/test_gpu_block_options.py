"""What a conditioned block's operators take beside the plain call, against the definitions in 64 bits, with the tolerances of
tests/test_gpu_block.py: the norms around a branch over few rows, many rows (teams with a ring) and long rows, with every kind,
gate and absent part; attention of a scale of 0."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from oracle import tokens
from tests._tokens import KINDS, TINY, UNIT, block_norm, cross_attention, done, f64, strided
from tests.test_gpu_block import check_block, check_cross_result
from tests.test_gpu_tokens import assert_within


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


# ---------------------------------------------------------------- factors that no product of two of them holds
def rare_rows(t, n, kind, post, pre, columns, alpha=1.0, beta=1.0, gates=True):
    """(sum, y) and their definitions for normal values, but for `columns`: [{name: value}, ..] from the first on."""
    x, r = strided((t, n), kind, 1, scale=2.0), strided((t, n), "fp32", 2)
    named = {k: strided((n,), kind, i + 3, mean=1.0) for i, k in enumerate(("post_weight", "pre_weight", "post_bias", "pre_bias"))}
    count = 3
    named.update({k: strided((count, n), kind, i + 8) for i, k in enumerate(("gate", "scale", "shift"))})
    for c, values in enumerate(columns):
        for k, v in values.items():
            (x if k == "x" else named[k])[..., c] = v
    gate, scale, shift = (named[k] for k in ("gate", "scale", "shift"))
    gate = gate if gates else None
    per = (t + count - 1) // count
    m = np.arange(t) // per
    s, y = torch.empty(t, n, device="cuda"), torch.empty_like(x)
    vectors = [named[k] for k in ("post_weight", "post_bias", "pre_weight", "pre_bias")]
    block_norm(x, r, s, y, post, *vectors[:2], pre, *vectors[2:], 1e-5, gate, "plain", scale, shift, None, per, count, alpha, beta,
               kind, "fp32")
    done()
    pw, pb, qw, qb = (f64(v) for v in vectors)
    with np.errstate(all="ignore"):
        ref = tokens.block_norm(f64(x), f64(r), post, pw, pb, pre, qw, qb, 1e-5, None if gate is None else f64(gate)[m], "plain",
                                f64(scale)[m], f64(shift)[m], alpha, beta)
    return (s, "fp32", ref[0], ref[2]), (y, kind, ref[1], ref[3])


def assert_rare(results, first):
    """Values within the tolerance, infinities and NaN where the definition has them; the `first` columns hold what the test is
    about.  The largest value is (2 - 2 UNIT) 2^127, so that infinities begin half a step above it, at (2 - UNIT) 2^127; what
    lies within fp32's losses of that border may go either way."""
    for out, kind, ref, size in results:
        border = (2 - UNIT[kind]) * 2.0 ** 127
        with np.errstate(invalid="ignore"):
            ref = np.where(np.abs(ref) >= border, np.copysign(np.inf, ref), ref)
            either = np.abs(np.abs(ref) / border - 1) < 2.0 ** -16
        got = np.where(either, ref, f64(out))
        fine = np.isfinite(ref)
        assert np.array_equal(got[~fine], ref[~fine], equal_nan=True), (got[:2, :first], ref[:2, :first])
        assert_within(got[fine], ref[fine], (UNIT[kind] * np.abs(ref) + TINY[kind] + 96 * 2.0 ** -24 * size)[fine])


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("t", [5, 700])
@pytest.mark.parametrize("n", WIDTHS)
def test_gates_whose_products_leave_fp32(t, n, kind):
    """(post(x) gate beta, a factor after the other: infinite gates, factors of 0 beside them, products
    of two vectors or of a gate and the branch's scale that are too large or too small while the value is neither."""
    inf, nan = float("inf"), float("nan")
    columns = [dict(gate=inf, post_weight=1.0, post_bias=-3.0), dict(gate=-inf, post_weight=0.0, post_bias=2.0),
               dict(gate=inf, post_weight=0.0, post_bias=0.0), dict(gate=1e25, post_weight=1e-30, post_bias=0.0),
               dict(gate=1e-25, post_weight=1e-20, post_bias=1e20), dict(gate=0.0, post_weight=1e30, post_bias=0.0),
               dict(gate=nan), dict(gate=0.0, post_weight=inf), dict(gate=1e-20, post_weight=1e30, post_bias=0.0)]
    for beta in (1.0, 1e20, 1e-25):
        assert_rare(rare_rows(t, n, kind, "rms", "none", columns, beta=beta), len(columns))
    # without a norm: values beside which only the gate's product with beta is off
    columns = [dict(x=1e-30, gate=1e30), dict(x=1e30, gate=1e-30), dict(x=inf, gate=-2.0), dict(x=-inf, gate=0.0)]
    for beta in (1.0, 1e30, 1e-25):
        assert_rare(rare_rows(t, n, kind, "none", "none", columns, beta=beta), len(columns))


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("t", [5, 700])
@pytest.mark.parametrize("n", WIDTHS)
def test_modulations_whose_products_leave_fp32(t, n, kind):
    """pre(s) (1 + scale) + shift: infinite scales, weights and biases, values of infinity under a negative scale, weights whose
    product with 1 + scale is too large."""
    inf = float("inf")
    columns = [dict(scale=inf, pre_weight=1.0, pre_bias=-3.0), dict(scale=-inf, pre_weight=0.0, pre_bias=1.0),
               dict(scale=-0.5, pre_weight=inf, pre_bias=0.0), dict(scale=-1.0), dict(scale=-0.5, pre_bias=inf),
               dict(shift=inf), dict(scale=1.0, pre_weight=3e38, pre_bias=0.0), dict(scale=-1.0, pre_weight=inf)]
    assert_rare(rare_rows(t, n, kind, "none", "rms", columns, gates=False), len(columns))
    columns = [dict(x=inf, scale=-0.5), dict(x=-inf, scale=-3.0), dict(x=inf, scale=-1.0), dict(scale=inf), dict(x=3e38, scale=1.0)]
    assert_rare(rare_rows(t, n, kind, "none", "none", columns, gates=False), len(columns))


@pytest.mark.parametrize("n", WIDTHS)
def test_rows_around_one_group_of_an_infinite_gate(n):
    """One group of four with a gate of infinity, rows of all groups and padding mixed, in place: each row as it is defined,
    padding as it was."""
    t, count = 700, 4
    m = np.random.default_rng(n).integers(-1, count + 1, t)
    x, r = strided((t, n), "bf16", 1), strided((t, n), "fp32", 2)
    w, b, gate, shift = strided((n,), "bf16", 3), strided((n,), "bf16", 4), strided((count, n), "bf16", 5), strided((count, n), "bf16", 6)
    gate[2, n // 2], b[n // 2] = float("inf"), -0.5
    use = (m >= 0) & (m < count)
    at = np.where(use, m, 0)
    with np.errstate(all="ignore"):
        s, y, size_s, size_y = tokens.block_norm(f64(x), f64(r), "rms", f64(w), f64(b), "none", None, None, 1e-5, f64(gate)[at], "plain",
                                                 None, f64(shift)[at], 1.0, 1.0)
    s[~use], y[~use], size_s[~use], size_y[~use] = f64(r)[~use], f64(x)[~use], 0, 0
    block_norm(x, r, r, x, "rms", w, b, "none", None, None, 1e-5, gate, "plain", None, shift,
               torch.tensor(m, dtype=torch.int32, device="cuda"), 0, count, 1.0, 1.0, "bf16", "fp32")
    done()
    assert np.isinf(s[at == 2][:, n // 2]).any()
    assert_rare(((r, "fp32", s, size_s), (x, "bf16", y, size_y)), 4)


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("tq", [1, 400])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_of_scale_0_weighs_keys_alike_however_large_their_products(tq, d):
    q, k = strided((2, tq, 4, d), "bf16", 1, scale=1e18), strided((2, 190, 2, d), "bf16", 2, scale=1e18)
    v = strided((2, 190, 2, d), "bf16", 3)
    o, lse = torch.empty_like(q), torch.empty(2, 4, tq, device="cuda")
    cross_attention(q, k, v, o, lse, None, None, None, 0.0, "bf16")
    done()
    ref = tokens.cross_attention(f64(q), f64(k), f64(v), [tq] * 2, [190] * 2, None, 0.0)
    check_cross_result(f64(o), lse, *ref, "bf16", d, 190)


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("tq,kv", [(1, 300), (1, 20000), (300, 200)])
def test_attention_with_one_operand_off_16_bytes(tq, kv, which):
    """Queries, keys, values or the output alone start a value further on: it alone is copied."""
    q, k, v, o = (strided((2, n, h, 64), "fp16", i, None, int(i == which)) for i, (n, h) in enumerate(((tq, 4), (kv, 2), (kv, 2), (tq, 4))))
    base = o._base.clone()
    lse = torch.empty(2, 4, tq, device="cuda")
    cross_attention(q, k, v, o, lse, None, None, None, 0.125, "fp16")
    done()
    ref = tokens.cross_attention(f64(q), f64(k), f64(v), [tq] * 2, [kv] * 2, None, 0.125)
    check_cross_result(f64(o), lse, *ref, "fp16", 64, kv)
    assert torch.equal(o._base[:int(which == 3)].view(torch.int16), base[:int(which == 3)].view(torch.int16))


# ---------------------------------------------------------------- graph capture
CAPTURE = """
import sys
sys.path.insert(0, {root!r})
import torch
from tests._tokens import done, strided, norm_rope
from tests.test_gpu_block import calls_of_every_form

calls = calls_of_every_form()
q, k = strided((3, 4, 64), "bf16", 5), strided((3, 2, 64), "bf16", 6)
norm_rope(q, q, k, k, None, None, None, None, 1e-6, None, None, None, None, 0, False, "bf16")  # the one call on the device
done()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for call, _ in calls:
        call()
for _ in range(2):
    graph.replay()
    torch.cuda.synchronize()
    got = [[t.clone() for t in outs] for _, outs in calls]
    for _, outs in calls:
        for t in outs:
            t.zero_()
for (call, outs), ref in zip(calls, got):
    call()
    done()
    assert all(a.any() and torch.equal(a, b) for a, b in zip(outs, ref))
print("captured")
"""


def test_every_form_of_a_block_can_be_captured_once_any_call_has_been_made():
    """In a process of its own, whose one call before the capture is a norm of heads."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", CAPTURE.format(root=root)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "captured" in run.stdout, run.stderr[-2000:]
