"""The token operators against their definitions in 64 bits (oracle/tokens.py).

Tolerances, per value: one rounding of the result (UNIT |y|), plus what fp32 arithmetic can lose on the way, from the
number of operations and the magnitudes that they work on:
  linear     k + 8 sums of products, each off by at most 2^-23 of the magnitudes added so far (a product may be cut, not
             rounded, when it is added), times 1.13, the steepest slope of the activations, and 2^-20 for their own error;
  norm       the mean over d values, root, weight, and two products: (d / 2 + 16) 2^-24 of the pair's magnitudes;
  attention  scores off by (d + 8) 2^-23 of the largest sum |q||k| and 2^-20 of their own, an exponential of 2^-20, and
             weights that are rounded to the storage type before their product with v: all of sum p |v|.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from oracle import tokens
from tests._tokens import (ACTS, KINDS, TINY, UNIT, attention, done, f64, linear, norm_rope, strided)

import conv2d_implicit_gemm_gb300 as ox


def assert_within(got, ref, tol):
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape
    off = np.abs(got - ref)
    bad = ~(off <= tol)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} values; worst {np.nanmax(off / np.maximum(tol, 1e-300)):.3g} times "
                           f"the tolerance; first at {np.argwhere(bad)[0]}: {got[tuple(np.argwhere(bad)[0])]} for "
                           f"{ref[tuple(np.argwhere(bad)[0])]}")


# ---------------------------------------------------------------- linear
def check_linear(m, n, k, kind, act="none", bias=True, residual=True, pad=0, shift=0, seed=0, inplace=False):
    x = strided((m, k), kind, seed, [0, pad], shift)
    w = strided((n, k), kind, seed + 1, [0, pad], shift, scale=1 / max(k, 1) ** 0.5)
    b = strided((n,), kind, seed + 2, None, shift) if bias else None
    r = strided((m, n), kind, seed + 3, [0, pad], shift) if residual else None
    ref, size = tokens.linear(f64(x), f64(w), f64(b), f64(r), act)
    y = r if inplace else strided((m, n), kind, seed + 4, [0, pad], shift)
    around = y.clone()
    base = y._base if y._base is not None else y
    outside = base.clone()
    linear(x, w, b, r, y, act, kind)
    done()
    tol = UNIT[kind] * np.abs(ref) + TINY[kind] + 1.13 * (k + 8) * 2.0 ** -23 * size + 2.0 ** -20 * np.abs(ref)
    if residual:
        tol = tol + 2.0 ** -23 * np.abs(ref)
    assert_within(f64(y), ref, tol)
    # nothing is written around the matrix
    y.copy_(around)
    assert torch.equal(base.view(torch.int16), outside.view(torch.int16))


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("m", [1, 2, 5, 8, 16, 17, 33, 64, 65, 128, 129, 257, 300])
def test_linear_rows(m, kind):
    check_linear(m, 264, 200, kind, "gelu", seed=m)


@pytest.mark.parametrize("n,k", [(1, 1), (1, 8), (8, 1), (7, 3), (16, 16), (127, 64), (129, 72), (256, 999), (1001, 8),
                                 (320, 2056), (40, 4104)])
@pytest.mark.parametrize("m", [1, 13, 70, 200])
def test_linear_odd_sizes(m, n, k):
    check_linear(m, n, k, "bf16" if (m + n) % 2 else "fp16", "silu", seed=n)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("m", [3, 150])
def test_linear_epilogues(m, act, bias, residual):
    check_linear(m, 136, 96, "fp16", act, bias, residual, seed=5)


@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (8, 1), (3, 0), (0, 1), (1, 2), (24, 4)])
@pytest.mark.parametrize("m", [1, 40, 140])
def test_linear_strides_and_alignment(m, pad, shift):
    check_linear(m, 144, 128, "bf16", "relu", pad=pad, shift=shift, seed=9)
    check_linear(m, 144, 129, "fp16", "none", pad=pad, shift=shift, seed=9)


@pytest.mark.parametrize("m", [1, 20, 130])
def test_linear_adds_to_its_residual_in_place(m):
    check_linear(m, 200, 64, "fp16", "gelu_tanh", inplace=True)
    check_linear(m, 201, 64, "bf16", "none", inplace=True)


@pytest.mark.parametrize("at", [(0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("m,n", [(140, 1), (140, 2), (140, 33), (150, 64), (600, 777), (2100, 2905)])
def test_linear_outputs_and_residuals_on_odd_places(m, n, at):
    """Rows of the output and of the residual that start on odd places, each in its own way."""
    x, w = strided((m, 72), "fp16", 1), strided((n, 72), "fp16", 2, scale=0.1)
    r, y = strided((m, n), "fp16", 3, [0, 2], at[0]), strided((m, n), "fp16", 4, [0, 3], at[1])
    around, outside = y.clone(), y._base.clone()
    ref, size = tokens.linear(f64(x), f64(w), None, f64(r), "none")
    linear(x, w, None, r, y, "none", "fp16")
    done()
    assert_within(f64(y), ref, UNIT["fp16"] * np.abs(ref) + TINY["fp16"] + 100 * 2.0 ** -23 * size + 2.0 ** -22 * np.abs(ref))
    base = y._base
    y.copy_(around)
    assert torch.equal(base.view(torch.int16), outside.view(torch.int16))


def test_linear_large_odd_sizes_in_place():
    check_linear(1500, 1501, 264, "bf16", "gelu_tanh", inplace=True, seed=6)
    check_linear(2100, 2999, 100, "fp16", "relu", inplace=True, seed=7)


def test_linear_large_tiles():
    check_linear(515, 777, 320, "bf16", "gelu_tanh", seed=3)
    check_linear(1100, 2048, 520, "fp16", "silu", residual=False, seed=4)
    check_linear(2300, 1032, 264, "bf16", "relu", seed=5)


@pytest.mark.parametrize("m", [2, 200])
def test_linear_without_products_is_the_epilogue(m):
    b, r = strided((50,), "fp16", 1), strided((m, 50), "fp16", 2)
    y = torch.empty(m, 50, dtype=torch.float16, device="cuda")
    ox.oidnx_linear(0, 0, 0, 0, b.data_ptr(), r.data_ptr(), 50, y.data_ptr(), 50, m, 50, 0, ox.ACT_RELU,
                    ox.PRECISION_FP16, torch.cuda.current_stream().cuda_stream)
    done()
    ref = np.maximum(f64(b), 0)[None] + f64(r)
    assert_within(f64(y), ref, UNIT["fp16"] * np.abs(ref) + 2.0 ** -23 * np.abs(ref) + TINY["fp16"])


def test_linear_without_products_of_very_many_rows():
    m = 65535 * 32 + 70  # more than one grid
    r = torch.randn(m, 2, device="cuda").half()
    y = torch.empty_like(r)
    ox.oidnx_linear(0, 0, 0, 0, 0, r.data_ptr(), 2, y.data_ptr(), 2, m, 2, 0, ox.ACT_NONE, ox.PRECISION_FP16,
                    torch.cuda.current_stream().cuda_stream)
    done()
    assert torch.equal(y, r)


@pytest.mark.parametrize("m", [4, 180])
def test_linear_infinities_and_nan_stay_in_their_rows_and_columns(m):
    x, w = strided((m, 64), "bf16", 1), strided((80, 64), "bf16", 2)
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    w[7, 9] = float("inf")
    y = torch.empty(m, 80, dtype=torch.bfloat16, device="cuda")
    linear(x, w, None, None, y, "relu", "bf16")
    done()
    got = f64(y)
    assert np.isnan(got[1]).all()
    assert (np.isinf(got[2]) | np.isnan(got[2]) | (got[2] == 0)).all()
    assert not np.isfinite(got[0, 7]) or got[0, 7] == 0
    rows = [i for i in range(m) if i not in (1, 2)]
    cols = [j for j in range(80) if j != 7]
    ref, size = tokens.linear(f64(x)[rows], f64(w)[cols], act="relu")
    assert_within(got[np.ix_(rows, cols)], ref, UNIT["bf16"] * np.abs(ref) + 100 * 2.0 ** -23 * size)


# ---------------------------------------------------------------- norm and rotation
def check_norm(t, hq, hk, d, rot, interleaved, kind, weight=True, slots=True, values=True, pad=0, shift=0, seed=0):
    rng = np.random.default_rng(seed + 100)
    q, k = strided((t, hq, d), kind, seed, [0, 0, pad], shift), strided((t, hk, d), kind, seed + 1, [0, 1, pad], shift)
    v = strided((t, hk, d), kind, seed + 2, [0, 0, pad], shift) if values else None
    rows = t + 37 if slots else t
    qo = strided((t, hq, d), kind, seed + 3, [0, 0, pad], shift)
    ko = strided((rows, hk, d), kind, seed + 4, [0, 0, pad], shift)
    vo = strided((rows, hk, d), kind, seed + 5, [0, 0, pad], shift) if values else None
    kept_k, kept_v = f64(ko), f64(vo)
    qw = strided((d,), kind, seed + 6, mean=1.0, scale=0.2) if weight else None
    kw = strided((d,), kind, seed + 7, mean=1.0, scale=0.2) if weight else None
    table = rng.uniform(-3, 3, (50, rot // 2)).astype(np.float32)
    cos, sin = torch.from_numpy(np.cos(table)).cuda(), torch.from_numpy(np.sin(table)).cuda()
    at = rng.integers(0, 50, t).astype(np.int32)
    to = rng.permutation(rows)[:t].astype(np.int32) if slots else np.arange(t)
    if slots and t > 2:
        to[1], to[2] = -1, rows  # padding: dropped
    norm_rope(q, qo, k, ko, v, vo, qw, kw, 1e-5, cos if rot else None, sin if rot else None,
              torch.from_numpy(at).cuda() if rot else None, torch.from_numpy(to).cuda() if slots else None, rot,
              interleaved, kind)
    done()
    c, s = f64(cos)[at], f64(sin)[at]
    for x, w, got, row in ((q, qw, qo, np.arange(t)), (k, kw, ko, to)):
        ref, size = tokens.norm_rope(f64(x), f64(w), 1e-5, c, s, rot, interleaved)
        use = (row >= 0) & (row < got.shape[0])
        tol = UNIT[kind] * np.abs(ref) + TINY[kind] + (d / 2 + 16) * 2.0 ** -24 * size
        assert_within(f64(got)[row[use]], ref[use], tol[use])
    use = (to >= 0) & (to < rows)
    rest = np.setdiff1d(np.arange(rows), to[use])
    assert np.array_equal(f64(ko)[rest], kept_k[rest])
    if values:
        assert np.array_equal(f64(vo)[to[use]], f64(v)[use])
        assert np.array_equal(f64(vo)[rest], kept_v[rest])


@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("d", [8, 32, 64, 72, 128, 200, 256, 512])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_head_sizes(d, interleaved, kind):
    check_norm(5, 6, 3, d, d, interleaved, kind, seed=d)
    check_norm(3, 5, 5, d, d // 2 // 2 * 2, interleaved, kind, weight=False, seed=d)


@pytest.mark.parametrize("d,rot", [(1, 0), (2, 2), (5, 4), (33, 10), (128, 6), (96, 0), (130, 130)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_odd_heads(d, rot, interleaved):
    check_norm(4, 3, 2, d, rot, interleaved, "fp16", seed=1)
    check_norm(4, 3, 2, d, rot, interleaved, "fp32", seed=2)


@pytest.mark.parametrize("t,hq,hk", [(1, 1, 1), (1, 32, 8), (1, 100, 70), (300, 7, 7), (1025, 4, 1)])
@pytest.mark.parametrize("slots,values", [(True, True), (False, True), (True, False)])
def test_norm_tokens_and_heads(t, hq, hk, slots, values):
    check_norm(t, hq, hk, 64, 64, False, "bf16", slots=slots, values=values, seed=t)


@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (3, 0), (0, 1), (8, 4)])
def test_norm_strides_and_alignment(pad, shift):
    check_norm(9, 4, 2, 64, 32, False, "fp16", pad=pad, shift=shift)
    check_norm(9, 4, 2, 64, 32, True, "fp32", pad=pad, shift=shift)


@pytest.mark.parametrize("d", [128, 65])
def test_norm_in_place(d):
    q, k = strided((10, 4, d), "bf16", 1), strided((10, 2, d), "bf16", 2)
    rot = d // 2 * 2
    cos = torch.full((10, rot // 2), 0.6, device="cuda")
    sin = torch.full((10, rot // 2), 0.8, device="cuda")
    at = torch.arange(10, dtype=torch.int32, device="cuda")
    refs = [tokens.norm_rope(f64(x), None, 0.0, f64(cos), f64(sin), rot, False) for x in (q, k)]
    norm_rope(q, q, k, k, None, None, None, None, 0.0, cos, sin, at, None, rot, False, "bf16")
    done()
    for x, (ref, size) in zip((q, k), refs):
        assert_within(f64(x), ref, UNIT["bf16"] * np.abs(ref) + (d / 2 + 16) * 2.0 ** -24 * size)


@pytest.mark.parametrize("d", [64, 65])
def test_norm_positions_outside_the_table_give_nan(d):
    q, k = strided((4, 2, d), "fp16", 1), strided((4, 2, d), "fp16", 2)
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    cos, sin = torch.ones(3, 16, device="cuda"), torch.zeros(3, 16, device="cuda")
    at = torch.tensor([0, -1, 3, 2], dtype=torch.int32, device="cuda")
    norm_rope(q, qo, k, ko, None, None, None, None, 1e-6, cos, sin, at, None, 32, False, "fp16")
    done()
    for got in (f64(qo), f64(ko)):
        assert np.isnan(got[1:3, :, :32]).all() and np.isfinite(got[1:3, :, 32:]).all()
        assert np.isfinite(got[[0, 3]]).all()


def test_norm_of_zeros_is_zero():
    q, k = (torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qo, ko = q + 1, k + 1
    norm_rope(q, qo, k, ko, None, None, None, None, 1e-6, None, None, None, None, 0, False, "bf16")
    done()
    assert not qo.any() and not ko.any()


# ---------------------------------------------------------------- attention
def check_attention(b, tq, cap, hq, hk, d, window, sinks, kind, q_lens=None, kv_lens=None, pad=0, shift=0, seed=0,
                    scale=None, size=1.0, edit=None, rows=None):
    q = strided((b, tq, hq, d), kind, seed, [0, 0, 0, pad], shift, scale=size)
    k = strided((b, cap, hk, d), kind, seed + 1, [0, 0, 1, pad], shift, scale=size)
    v = strided((b, cap, hk, d), kind, seed + 2, [1, 0, 0, pad], shift)
    ql = np.full(b, tq) if q_lens is None else np.array(q_lens)
    kl = np.full(b, cap) if kv_lens is None else np.array(kv_lens)
    for s in range(b):  # what no key was written to
        k[s, min(kl[s], cap):] = float("nan")
        v[s, min(kl[s], cap):] = float("inf")
    if edit:
        edit(q, k, v)
    o = strided((b, tq, hq, d), kind, seed + 3, [0, 0, 0, pad], shift)
    lse = torch.full((b, hq, tq), 7.0, device="cuda")
    scale = d ** -0.5 if scale is None else scale
    attention(q, k, v, o, lse, None if q_lens is None else torch.tensor(ql, dtype=torch.int32, device="cuda"),
              None if kv_lens is None else torch.tensor(kl, dtype=torch.int32, device="cuda"), window, sinks, scale, kind)
    done()
    ref, ref_lse, mag, dots = tokens.window_attention(f64(q), f64(k), f64(v), ql, kl, window, sinks, scale)
    if rows is not None:
        return f64(o), ref, mag
    score = (d + 8) * 2.0 ** -23 * dots + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(ref_lse), ref_lse, 0)).max())
    most = float(np.nanmax(np.abs(f64(v)), where=np.isfinite(f64(v)), initial=0))
    tol = (UNIT[kind] * np.abs(ref) + TINY[kind] + (2 * UNIT[kind] + 4 * score + 2.0 ** -18) * mag
           + TINY[kind] * 2 * cap * most)
    assert_within(f64(o), ref, tol)
    got = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(got), np.isneginf(ref_lse))
    fine = np.isfinite(ref_lse)
    assert_within(got[fine], ref_lse[fine], np.full(fine.sum(), 2 * score + 2.0 ** -18))
    empty = ~fine.transpose(0, 2, 1)
    assert (f64(o)[empty] == 0).all()


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [8, 40, 64, 80, 128])
@pytest.mark.parametrize("tq,cap", [(1, 1), (1, 300), (3, 129), (40, 40), (130, 200), (200, 333)])
def test_attention_sizes(tq, cap, d, kind):
    check_attention(2, tq, cap, 4, 2, d, 50, 3, kind, seed=d)


@pytest.mark.parametrize("d", [1, 20, 63, 100, 136, 200, 256])
@pytest.mark.parametrize("tq", [1, 30])
def test_attention_odd_heads(tq, d):
    check_attention(1, tq, 70, 2, 1, d, 20, 2, "fp16", seed=d)


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 5), (1, 0), (1, 1), (7, 200), (64, 4), (127, 0), (128, 128),
                                          (129, 1), (1000, 1000), (2147483647, 3)])
@pytest.mark.parametrize("tq,cap", [(1, 400), (5, 400), (400, 400), (137, 390)])
def test_attention_windows_and_sinks(tq, cap, window, sinks):
    check_attention(1, tq, cap, 2, 2, 64, window, sinks, "bf16", seed=window % 1000)


@pytest.mark.parametrize("hq,hk", [(1, 1), (7, 1), (8, 8), (32, 4), (40, 1), (6, 2)])
@pytest.mark.parametrize("tq", [1, 2, 9, 90])
def test_attention_shared_heads(tq, hq, hk):
    check_attention(2, tq, 150, hq, hk, 64, 100, 4, "fp16", seed=hq)


@pytest.mark.parametrize("tq", [1, 4, 33, 160])
@pytest.mark.parametrize("sinks,window", [(0, 0), (4, 30), (0, 64)])
def test_attention_ragged_lengths_and_empty_rows(tq, sinks, window):
    cap = 200
    check_attention(7, tq, cap, 4, 2, 72, window, sinks, "bf16", q_lens=[tq, tq, 0, max(1, tq // 2), tq, 1, tq],
                    kv_lens=[cap, 0, 50, 150, tq // 2, 1, 129], seed=tq)


@pytest.mark.parametrize("tq", [1, 3, 60])
@pytest.mark.parametrize("cap,sinks,window", [(100, 4, 30), (100, 0, 36), (257, 7, 0), (100, 4, 96), (100, 100, 20),
                                              (65, 64, 10), (130, 1, 500)])
def test_attention_ring_cache(tq, cap, sinks, window):
    check_attention(4, tq, cap, 2, 1, 64, window, sinks, "fp16",
                    kv_lens=[cap, cap + 1, 3 * cap + 17, 1000003], seed=cap)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tq,cap,kv,window,sinks", [
    (300, 2500, 2390, 900, 4), (200, 3000, 2871, 0, 0), (600, 1500, 1500, 700, 130), (150, 1400, 5000, 1200, 7),
    (90, 4000, 3980, 3000, 1)])
def test_attention_many_key_tiles(tq, cap, kv, window, sinks, d):
    """Long caches with partly written last tiles: first and last tiles masked, many whole ones between."""
    check_attention(2, tq, cap, 2, 1, d, window, sinks, "bf16", kv_lens=[kv, min(kv, cap) - 131], seed=kv)


@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (3, 0), (0, 1), (8, 4)])
@pytest.mark.parametrize("tq", [1, 70])
def test_attention_strides_and_alignment(tq, pad, shift):
    check_attention(2, tq, 140, 4, 2, 64, 60, 2, "bf16", pad=pad, shift=shift)


@pytest.mark.parametrize("tq", [1, 200])
@pytest.mark.parametrize("scale,size", [(1.0, 3.0), (0.0, 1.0), (-0.5, 1.0), (0.02, 12.0)])
def test_attention_sharp_and_flat_scores(tq, scale, size):
    check_attention(1, tq, 300, 2, 2, 64, 0, 0, "fp16", scale=scale, size=size, seed=3)


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [40, 64, 80, 128])
@pytest.mark.parametrize("tq", [1, 300, 690])
def test_attention_scores_that_grow_along_the_keys(tq, d, kind):
    """Every 64 keys are larger than those before: sums and outputs are scaled again and again."""
    def edit(q, k, v):
        k *= (1 + torch.arange(700, device="cuda") // 64 * 2).to(k.dtype)[None, :, None, None]

    check_attention(1, tq, 700, 4, 2, d, 0, 0, kind, edit=edit, seed=d + tq)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tq,window", [(600, 30), (600, 200), (257, 1)])
def test_attention_row_tiles_that_see_other_key_tiles(tq, window, d):
    """Row tiles next to each other whose windows share no key, over many pairs of them."""
    check_attention(3, tq, 1500, 2, 2, d, window, 0, "fp16", kv_lens=[1500, 700, 1111], seed=window)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attention_unseen_values_of_large_heads_and_long_caches(bad):
    """The same for heads of 128 values, whole key tiles before and after the one that holds the value."""
    at, tq, n, window = 1000, 900, 1600, 300

    def edit(q, k, v):
        v[0, at, 0, 100] = bad

    got, ref, mag = check_attention(1, tq, n, 4, 1, 128, window, 2, "bf16", edit=edit, rows=True, seed=9)
    pos = n - tq + np.arange(tq)
    sees = (at <= pos) & (at > pos - window)
    np.testing.assert_array_equal(np.isfinite(got[0][~sees]), True)
    assert not np.isfinite(got[0][sees][:, :, 100]).any()
    got, ref, mag = got[0].copy(), ref[0].copy(), mag[0].copy()
    got[sees, :, 100] = ref[sees, :, 100] = mag[sees, :, 100] = 0
    assert_within(got, ref, UNIT["bf16"] * np.abs(ref) + (2 * UNIT["bf16"] + 2.0 ** -14) * mag)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("tq", [1, 6, 300])
def test_attention_unseen_keys_never_reach_a_row(tq, bad):
    """A value that is no number sits at one key; only the rows that see the key are touched by it."""
    at = 350 - 20 if tq == 1 else 350 - tq + tq // 2

    def edit(q, k, v):
        v[0, at, 0, 5] = bad

    window = 10
    got, ref, mag = check_attention(1, tq, 350, 2, 1, 64, window, 2, "bf16", edit=edit, rows=True, seed=8)
    pos = 350 - tq + np.arange(tq)
    sees = (at <= pos) & (at > pos - window)
    np.testing.assert_array_equal(np.isfinite(got[0][~sees]), True)
    assert not np.isfinite(got[0][sees][:, :, 5]).any()
    got, ref, mag = got[0].copy(), ref[0].copy(), mag[0].copy()
    got[sees, :, 5] = ref[sees, :, 5] = mag[sees, :, 5] = 0
    assert_within(got, ref, UNIT["bf16"] * np.abs(ref) + (2 * UNIT["bf16"] + 2.0 ** -14) * mag)


@pytest.mark.parametrize("tq", [1, 200])
def test_attention_keys_that_are_no_numbers(tq):
    """A key that is NaN makes the rows that see it NaN and no other."""
    def edit(q, k, v):
        k[0, 240, 0, 3] = float("nan")

    got, ref, mag = check_attention(1, tq, 300, 2, 1, 64, 16, 0, "fp16", edit=edit, rows=True, seed=8)
    pos = 300 - tq + np.arange(tq)
    sees = (240 <= pos) & (240 > pos - 16)
    assert np.isnan(got[0][sees]).all()
    assert_within(got[0][~sees], ref[0][~sees],
                  (UNIT["fp16"] * np.abs(ref) + TINY["fp16"] * 600 + (2 * UNIT["fp16"] + 2.0 ** -14) * mag)[0][~sees])


@pytest.mark.parametrize("tq", [1, 90])
def test_attention_shared_keys_and_strides_of_single_elements(tq):
    """Keys and values broadcast over sequences and heads; dimensions of one element with strides that mean nothing."""
    q = strided((3, tq, 4, 64), "bf16", 1)
    k, v = (strided((1, 200, 1, 64), "bf16", i).expand(3, 200, 2, 64) for i in (2, 3))
    o, lse = torch.empty_like(q), torch.empty(3, 4, tq, device="cuda")
    attention(q, k, v, o, lse, None, None, 40, 2, 0.125, "bf16")
    done()
    ref, ref_lse, mag, dots = tokens.window_attention(f64(q), f64(k), f64(v), [tq] * 3, [200] * 3, 40, 2, 0.125)
    assert_within(f64(o), ref, UNIT["bf16"] * np.abs(ref) + (2 * UNIT["bf16"] + 2.0 ** -14) * mag)
    q1, k1, v1 = q[:1, :, :1], k[:1, :, :1].contiguous(), v[:1, :, :1].contiguous()
    o1 = torch.zeros(1, tq, 1, 64, dtype=torch.bfloat16, device="cuda")
    ox.oidnx_window_attention(q1.data_ptr(), 3, q1.stride(1), 5, k1.data_ptr(), 0, k1.stride(1), 1, v1.data_ptr(), -7,
                              v1.stride(1), 9, o1.data_ptr(), 11, o1.stride(1), 13, 0, 0, 0, 1, tq, 200, 1, 1, 64, 40, 2,
                              0.125, ox.PRECISION_BF16, torch.cuda.current_stream().cuda_stream)
    done()
    assert_within(f64(o1), ref[:1, :, :1], (UNIT["bf16"] * np.abs(ref) + (2 * UNIT["bf16"] + 2.0 ** -14) * mag)[:1, :, :1])


def test_attention_many_sequences_of_single_tokens():
    rng = np.random.default_rng(4)
    check_attention(90, 1, 260, 8, 2, 128, 100, 4, "bf16", kv_lens=rng.integers(0, 600, 90), seed=6)


def test_attention_long_cache_beyond_32_bit_offsets():
    """A cache of over 2^31 elements: the last slots are read where they are."""
    cap, hk, d = 2 ** 31 // 512 + 4096, 4, 128
    k = torch.zeros(1, cap, hk, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    tail = strided((1, 300, hk, d), "bf16", 1)
    k[:, -300:], v[:, -300:] = tail, tail.flip(1)
    v[:, :300] = 1.0
    for tq in (1, 150):
        q = strided((1, tq, hk, d), "bf16", 2)
        o, lse = torch.empty_like(q), torch.empty(1, hk, tq, device="cuda")
        attention(q, k, v, o, lse, None, None, 100, 0, d ** -0.5, "bf16")
        done()
        ref, ref_lse, mag, dots = tokens.window_attention(f64(q), f64(k[:, -300:]), f64(v[:, -300:]), [tq], [300], 100, 0,
                                                          d ** -0.5)
        assert_within(f64(o), ref, UNIT["bf16"] * np.abs(ref) + (2 * UNIT["bf16"] + 2.0 ** -14) * mag)
        assert_within(lse.double().cpu().numpy(), ref_lse, np.full(ref_lse.shape, 2.0 ** -14))


# ---------------------------------------------------------------- all of them
def test_results_do_not_depend_on_the_stream_or_on_what_ran_before():
    x, w = strided((70, 520), "fp16", 1), strided((512, 520), "fp16", 2)
    q, k = strided((2, 5, 8, 64), "fp16", 3), strided((2, 900, 2, 64), "fp16", 4)
    first = None
    side = torch.cuda.Stream()
    for s in (torch.cuda.current_stream(), side, side):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            y = torch.empty(70, 512, dtype=torch.float16, device="cuda")
            o, lse = torch.empty_like(q), torch.empty(2, 8, 5, device="cuda")
            linear(x, w, None, None, y, "gelu", "fp16")
            attention(q, k, k, o, lse, None, None, 300, 4, 0.125, "fp16")
            done()
            got = [t.clone() for t in (y, o, lse)]
        s.synchronize()
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))


@pytest.mark.parametrize("hq,hk,d", [(6, 2, 80), (3, 1, 64), (7, 1, 128), (5, 1, 40)])
def test_attention_bits_do_not_depend_on_what_shared_memory_held(hq, hk, d):
    """Groups that do not fill a row tile: the same bits with other calls in between."""
    q, k, v = strided((2, 160, hq, d), "fp16", 1), strided((2, 900, hk, d), "fp16", 2), strided((2, 900, hk, d), "fp16", 3)
    loud = [strided((2, 200, 4, n), "fp16", 4, scale=30.0) for n in (64, 128)]

    def call():
        o, lse = torch.empty_like(q), torch.empty(2, hq, 160, device="cuda")
        attention(q, k, v, o, lse, None, None, 400, 2, d ** -0.5, "fp16")
        return o, lse

    first = call()
    for _ in range(10):
        for x in loud:
            attention(x, x, x, torch.empty_like(x), None, None, None, 0, 0, 1.0, "fp16")
        again = call()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    done()


def test_calls_can_be_captured_into_a_graph():
    x, w = strided((9, 256), "bf16", 1), strided((256, 256), "bf16", 2)
    xo, wo = strided((200, 255), "bf16", 5), strided((64, 255), "bf16", 6)  # laid out anew in memory of the call
    yo = torch.empty(200, 64, dtype=torch.bfloat16, device="cuda")
    q, k = strided((1, 1, 8, 64), "bf16", 3), strided((1, 900, 2, 64), "bf16", 4)
    y, o = torch.empty(9, 256, dtype=torch.bfloat16, device="cuda"), torch.empty_like(q)

    def step():
        linear(x, w, None, None, y, "silu", "bf16")
        linear(xo, wo, None, None, yo, "none", "bf16")
        attention(q, k, k, o, None, None, None, 300, 4, 0.125, "bf16")

    step()
    done()
    ref = [y.clone(), o.clone(), yo.clone()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    y.zero_(), o.zero_(), yo.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, ref[0]) and torch.equal(o, ref[1]) and torch.equal(yo, ref[2])


def test_calls_from_a_thread_of_its_own():
    import threading
    x, w = strided((9, 256), "bf16", 1), strided((64, 256), "bf16", 2)
    y = torch.empty(9, 64, dtype=torch.bfloat16, device="cuda")
    ref = torch.empty_like(y)
    linear(x, w, None, None, ref, "none", "bf16")
    done()
    args = (x.data_ptr(), 256, w.data_ptr(), 256, 0, 0, 0, y.data_ptr(), 64, 9, 64, 256, ox.ACT_NONE, ox.PRECISION_BF16,
            torch.cuda.current_stream().cuda_stream)
    failed = []

    def work():
        try:
            ox.oidnx_linear(*args)
        except Exception as e:
            failed.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    done()
    assert not failed and torch.equal(y, ref)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_stream_in_steps_over_a_ring_equals_one_pass(dtype):
    """The example's block: prompt steps, then single tokens, over a ring, against one call over a cache of everything.
    The two round the same intermediate values to 16 bits in places that differ by what fp32 sums in another order give:
    a few units of the storage type through six roundings."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_stream.py")
    spec = importlib.util.spec_from_file_location("attention_stream", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    off = example.run(tokens=450, prompt_step=48, singles=12, streams=3, window=100, dtype=dtype, channels=256)
    assert off <= 6 * UNIT["fp16" if dtype == torch.float16 else "bf16"]
