"""A conditioned block's operators against their definitions in 64 bits (oracle/tokens.py).

Tolerances, per value: one rounding of the result (UNIT |y|), plus what fp32 arithmetic can lose on the way:
  block norm  a thread adds up to 32 values and their sums go through a tree of 5 + 16: sums are off by 53 2^-24 of what
              they add, roots by half of that, and ten operations on a value by 2^-24 each: 96 2^-24 of the magnitudes that
              the oracle carries along (a tanh or sigmoid by 2^-22: 4 more).  Rows of more than 16384 values add 256 at a time:
              512 2^-24;
  axes        as the norm and rotation of one axis: (d / 2 + 16) 2^-24 of the pair's magnitudes;
  attention   as that with a window: scores off by (d + 8) 2^-23 of the largest sum |q||k| and 2^-20 of their own, an
              exponential of 2^-20, and weights rounded to the storage type before their product with v: all of sum p |v|.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from oracle import tokens
from tests._tokens import (KINDS, TINY, UNIT, block_norm, cross_attention, done, f64, norm_rope, norm_rope_axes, strided)
from tests.test_gpu_tokens import assert_within


# ---------------------------------------------------------------- norms around a branch
def check_block(t, n, kind, total_kind=None, post="rms", pre="rms", gate="groups", gate_act="plain", scale=True, shift=True,
                bias=True, weight=True, residual=True, total=True, y=True, per=None, count=None, groups=None, alpha=1.0,
                beta=1.0, pad=0, shift_at=0, seed=0, inplace=False, mean=0.3, eps=1e-5):
    total_kind = total_kind or kind
    per = max(1, t) if per is None else per
    count = count if count is not None else (t + per - 1) // per

    def vector(i, **how):
        return strided((n,), kind, seed + i, None, shift_at, **how)

    x = strided((t, n), kind, seed, [0, pad], shift_at, scale=2.0, mean=mean)
    r = strided((t, n), total_kind, seed + 1, [0, pad], shift_at, scale=3.0, mean=mean) if residual else None
    pw, qw = (vector(i, scale=0.2, mean=1.0) if weight else None for i in (2, 3))
    pb, qb = (vector(i, scale=0.5) if bias else None for i in (4, 5))
    rows = {"groups": count, "channel": 1}.get(gate)
    g = strided((rows, n), kind, seed + 6, [0, pad], shift_at) if rows else None
    given = g if g is None or gate == "groups" else g.expand(count, n)  # a stride of 0: one row for all
    sc = strided((count, n), kind, seed + 7, [0, pad], shift_at, scale=0.3) if scale else None
    sh = strided((count, n), kind, seed + 8, [0, pad], shift_at) if shift else None
    s_out = (r if inplace else strided((t, n), total_kind, seed + 9, [0, pad], shift_at)) if total else None
    y_out = (x if inplace else strided((t, n), kind, seed + 10, [0, pad], shift_at)) if y else None
    m = np.arange(t) // per if groups is None else np.array(groups)
    use = (m >= 0) & (m < count)
    at = np.where(use, m, 0)
    ref_s, ref_y, size_s, size_y = tokens.block_norm(
        f64(x), f64(r), post, f64(pw), f64(pb), pre, f64(qw), f64(qb), eps, None if g is None else f64(given)[at], gate_act,
        f64(sc)[at] if scale else None, f64(sh)[at] if shift else None, alpha, beta)
    kept = [(out, out.clone(), out._base, out._base.clone()) for out in (s_out, y_out) if out is not None]
    block_norm(x, r, s_out, y_out, post, pw, pb, pre, qw, qb, eps, given, gate_act, sc, sh,
               None if groups is None else torch.tensor(m, dtype=torch.int32, device="cuda"), per, count, alpha, beta, kind,
               total_kind)
    done()
    loss = (512 if n > 16384 else 96 + (4 if gate_act != "plain" else 0)) * 2.0 ** -24
    for out, ref, size, k in ((s_out, ref_s, size_s, total_kind), (y_out, ref_y, size_y, kind)):
        if out is not None:
            assert_within(f64(out)[use], ref[use], (UNIT[k] * np.abs(ref) + TINY[k] + loss * size)[use])
    # padding rows and what lies between the rows stay as they were
    for out, before, base, base_before in kept:
        assert torch.equal(out[torch.tensor(~use)].cpu().view(torch.uint8), before[torch.tensor(~use)].cpu().view(torch.uint8))
        out.copy_(before)
        assert torch.equal(base.view(torch.uint8), base_before.view(torch.uint8))


@pytest.mark.parametrize("kind,total_kind", [("fp16", "fp16"), ("bf16", "bf16"), ("fp32", "fp32"), ("fp16", "fp32"),
                                             ("bf16", "fp32")])
@pytest.mark.parametrize("n", [8, 248, 256, 512, 1000, 1024, 2048, 4096, 8192, 16384, 16400])
def test_block_norm_widths(n, kind, total_kind):
    check_block(5, n, kind, total_kind, per=2, seed=n)


@pytest.mark.parametrize("kind,total_kind", [("fp16", "fp16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("n", [1, 2, 7, 33, 255, 257, 999, 1025, 4095, 4097, 16383, 16385, 40001])
def test_block_norm_odd_widths(n, kind, total_kind):
    check_block(4, n, kind, total_kind, post="layer", pre="layer", per=3, seed=n)


@pytest.mark.parametrize("n", [64, 1001, 2048, 5000, 17000])
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
def test_block_norm_kinds(n, post, pre):
    check_block(3, n, "bf16", "fp32", post=post, pre=pre, per=1, alpha=0.7, beta=-1.3, seed=n)


@pytest.mark.parametrize("gate", ["none", "channel", "groups"])
@pytest.mark.parametrize("gate_act", ["plain", "tanh", "sigmoid"])
@pytest.mark.parametrize("n", [96, 333, 17000])
def test_block_norm_gates(n, gate, gate_act):
    check_block(6, n, "fp16", gate=gate, gate_act=gate_act, per=4, seed=n)


@pytest.mark.parametrize("n", [128, 77, 3000, 20000])
@pytest.mark.parametrize("without", ["scale", "shift", "bias", "weight", "residual", "total", "y"])
def test_block_norm_without_its_parts(n, without):
    check_block(4, n, "bf16", **{without: False}, per=3, seed=n)


@pytest.mark.parametrize("t", [1, 2, 3, 4, 5, 152, 153, 3000])
@pytest.mark.parametrize("n", [72, 1500, 4096])
def test_block_norm_rows(t, n):
    check_block(t, n, "bf16", "fp32", per=max(1, t // 3), seed=t)


@pytest.mark.parametrize("pad,shift_at", [(8, 0), (8, 8), (8, 1), (3, 0), (0, 1), (4, 4)])
@pytest.mark.parametrize("n", [64, 1024, 4096, 20000])
def test_block_norm_strides_and_alignment(n, pad, shift_at):
    check_block(5, n, "fp16", per=2, pad=pad, shift_at=shift_at)


@pytest.mark.parametrize("pad,shift_at", [(0, 0), (8, 8), (3, 1)])
@pytest.mark.parametrize("n", [1, 8, 15, 16, 120, 128, 129, 136, 248, 256, 257, 264, 504, 512, 513, 520, 1024, 1025, 1032, 1544,
                               2600, 4104, 4609, 7680, 7681, 8191, 8192])
@pytest.mark.parametrize("kind,total_kind", [("fp16", "fp16"), ("bf16", "fp32"), ("fp32", "fp32")])
def test_block_norm_many_rows_of_each_width(n, pad, shift_at, kind, total_kind):
    """Rows of a part of a warp, of one warp, of two to sixteen, on and off 16 bytes."""
    check_block(641, n, kind, total_kind, post="layer", pre="rms", per=200, pad=pad, shift_at=shift_at, seed=n)


@pytest.mark.parametrize("n", [64, 1001, 4096, 17001])
@pytest.mark.parametrize("t", [3, 700])
def test_block_norm_in_place(n, t):
    check_block(t, n, "bf16", "fp32" if n == 4096 else "bf16", per=t, inplace=True)


@pytest.mark.parametrize("n", [64, 513, 4096, 17000])
def test_block_norm_leaves_padding_rows(n):
    check_block(9, n, "fp16", count=3, groups=[2, -1, 0, 3, 1, 1, 2 ** 31 - 1, -2 ** 31, 2])


def test_block_norm_leaves_padding_rows_of_many():
    rng = np.random.default_rng(3)
    check_block(5000, 256, "bf16", count=7, groups=rng.integers(-1, 8, 5000))


@pytest.mark.parametrize("n", [256, 3001, 20000])
def test_block_norm_of_rows_far_from_zero(n):
    """A mean a thousand times the deviation: the squares are those of what the mean leaves."""
    check_block(3, n, "fp32", post="layer", pre="layer", mean=1000.0, gate="none", scale=False, shift=False)


def test_block_norm_infinities_and_nan_stay_in_their_rows():
    x = strided((40, 200), "bf16", 1)
    y = torch.zeros_like(x)
    plain = torch.zeros_like(x)
    block_norm(x, None, None, plain, "none", None, None, "rms", None, None, 1e-6, None, "plain", None, None, None, 40, 1, 1.0, 1.0,
               "bf16", "bf16")
    x[7, 3], x[20, 0] = float("nan"), float("inf")
    block_norm(x, None, None, y, "none", None, None, "rms", None, None, 1e-6, None, "plain", None, None, None, 40, 1, 1.0, 1.0,
               "bf16", "bf16")
    done()
    rest = [i for i in range(40) if i not in (7, 20)]
    assert torch.equal(y[rest], plain[rest])
    assert y[7].isnan().all() and y[20, 0].isnan()


def test_block_norm_beyond_32_bit_offsets():
    t, n = 2 ** 31 // 8192 + 5, 8192
    x = torch.zeros(t, n, dtype=torch.bfloat16, device="cuda")
    x[-1] = strided((n,), "bf16", 1)
    y = torch.empty_like(x)
    block_norm(x, None, None, y, "none", None, None, "rms", None, None, 1e-6, None, "plain", None, None, None, t, 1, 1.0, 1.0, "bf16",
               "bf16")
    done()
    _, ref, _, size = tokens.block_norm(f64(x[-1:]), None, "none", None, None, "rms", None, None, 1e-6, None, "plain", None,
                                        None, 1.0, 1.0)
    assert_within(f64(y[-1:]), ref, UNIT["bf16"] * np.abs(ref) + 96 * 2.0 ** -24 * size)
    assert not y[0].any() and not y[-2].any()


# ---------------------------------------------------------------- rotation by several axes
def check_axes(t, hq, hk, d, pair_axes, axes, interleaved, kind, norm=True, weight=True, slots=True, values=True, pad=0,
               shift=0, seed=0, outside=False):
    rng = np.random.default_rng(seed + 100)
    rot = 2 * len(pair_axes)
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
    at = rng.integers(0, 50, (axes, t)).astype(np.int32)
    if outside:
        at[0, ::3], at[axes - 1, 1::3] = -1, 50
    positions = torch.full((axes, t + 3), -9, dtype=torch.int32, device="cuda")[:, :t]
    positions.copy_(torch.from_numpy(at))
    to = rng.permutation(rows)[:t].astype(np.int32) if slots else np.arange(t)
    if slots and t > 2:
        to[1], to[2] = -1, rows  # padding: dropped
    norm_rope_axes(q, qo, k, ko, v, vo, norm, qw, kw, 1e-5, cos, sin, positions, pair_axes,
                   torch.from_numpy(to).cuda() if slots else None, interleaved, kind)
    done()
    c, s = tokens.axes_rows(f64(cos), at, pair_axes), tokens.axes_rows(f64(sin), at, pair_axes)
    for x, w, got, row in ((q, qw, qo, np.arange(t)), (k, kw, ko, to)):
        ref, size = tokens.norm_rope(f64(x), f64(w), 1e-5, c, s, rot, interleaved, norm)
        use = (row >= 0) & (row < got.shape[0])
        tol = UNIT[kind] * np.abs(ref) + TINY[kind] + (d / 2 + 16) * 2.0 ** -24 * size
        out, ref, tol = f64(got)[row[use]], ref[use], tol[use]
        assert np.array_equal(np.isnan(out), np.isnan(ref))
        fine = ~np.isnan(ref)
        assert_within(out[fine], ref[fine], tol[fine])
    use = (to >= 0) & (to < rows)
    rest = np.setdiff1d(np.arange(rows), to[use])
    assert np.array_equal(f64(ko)[rest], kept_k[rest])
    if values:
        assert np.array_equal(f64(vo)[to[use]], f64(v)[use])
        assert np.array_equal(f64(vo)[rest], kept_v[rest])


def sections(*counts):
    return [a for a, n in enumerate(counts) for _ in range(n)]


@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("d", [8, 32, 64, 72, 128, 200, 256, 512])
@pytest.mark.parametrize("interleaved", [False, True])
def test_axes_head_sizes(d, interleaved, kind):
    pairs = d // 2
    check_axes(11, 3, 2, d, sections(pairs // 3, pairs // 2, pairs - pairs // 3 - pairs // 2), 3, interleaved, kind, seed=d)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("axes", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("d,pairs", [(128, 64), (128, 32), (64, 32), (80, 40), (33, 10), (2, 1), (6, 0)])
def test_axes_in_turns(d, pairs, axes, kind):
    check_axes(7, 4, 2, d, [r % axes for r in range(pairs)], axes, False, kind, seed=d + axes)


@pytest.mark.parametrize("norm,weight", [(True, False), (False, False), (False, True)])
@pytest.mark.parametrize("d", [64, 128, 88, 65])
def test_axes_without_norm_or_weight(d, norm, weight):
    check_axes(9, 4, 4, d, sections(8, 12, 12), 3, True, "fp16", norm=norm, weight=weight, seed=d)


@pytest.mark.parametrize("t,hq,hk", [(1, 1, 1), (1, 32, 8), (1, 100, 70), (300, 7, 7), (1025, 4, 1), (4000, 8, 2)])
@pytest.mark.parametrize("slots,values", [(True, True), (False, True), (True, False)])
def test_axes_tokens_and_heads(t, hq, hk, slots, values):
    check_axes(t, hq, hk, 128, sections(16, 24, 24), 3, False, "bf16", slots=slots, values=values, seed=t)


@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (3, 0), (0, 1), (8, 4)])
def test_axes_strides_and_alignment(pad, shift):
    check_axes(21, 4, 2, 64, sections(10, 11, 11), 3, False, "fp16", pad=pad, shift=shift)


@pytest.mark.parametrize("d", [64, 66])
@pytest.mark.parametrize("turns", [False, True])
def test_axes_positions_outside_the_table_give_nan_to_their_pairs(d, turns):
    check_axes(30, 2, 2, d, [r % 3 for r in range(24)] if turns else sections(8, 8, 8), 3, False, "bf16", outside=True)


def test_axes_of_one_is_the_rotation_by_one_position():
    q, k, v = (strided((500, h, 128), "bf16", h) for h in (8, 2, 2))
    w = strided((128,), "bf16", 5, mean=1.0)
    table = torch.randn(600, 64, device="cuda")
    at = torch.randint(0, 600, (1, 500), dtype=torch.int32, device="cuda")
    one = [torch.empty_like(x) for x in (q, k, v)]
    other = [torch.empty_like(x) for x in (q, k, v)]
    norm_rope(q, one[0], k, one[1], v, one[2], w, w, 1e-6, table.cos(), table.sin(), at[0], None, 128, False, "bf16")
    norm_rope_axes(q, other[0], k, other[1], v, other[2], True, w, w, 1e-6, table.cos(), table.sin(), at, [0] * 64, None, False,
                   "bf16")
    done()
    for a, b in zip(one, other):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- attention to an encoder's states
def check_cross(b, tq, kv, hq, hk, d, kind, q_lens=None, kv_lens=None, mask=None, pad=0, shift=0, seed=0, scale=None, size=1.0,
                edit=None, with_lse=True):
    q = strided((b, tq, hq, d), kind, seed, [0, 0, 0, pad], shift, scale=size)
    k = strided((b, kv, hk, d), kind, seed + 1, [0, 0, 1, pad], shift, scale=size)
    v = strided((b, kv, hk, d), kind, seed + 2, [1, 0, 0, pad], shift)
    ql = np.full(b, tq) if q_lens is None else np.array(q_lens)
    kl = np.full(b, kv) if kv_lens is None else np.array(kv_lens)
    if edit:
        edit(q, k, v)
    given = None
    if mask is not None:
        mask = np.broadcast_to(mask, (b, kv))
        given = torch.full((b, kv + 5), 255, dtype=torch.uint8, device="cuda")[:, :kv]
        given.copy_(torch.from_numpy(mask.astype(np.uint8) * 3))
    for s in range(b):  # what is not seen holds anything
        k[s, kl[s]:] = float("nan")
        v[s, kl[s]:] = float("inf")
        if mask is not None:
            k[s, torch.from_numpy(mask[s] == 0).cuda()] = float("inf")
            v[s, torch.from_numpy(mask[s] == 0).cuda()] = float("nan")
    o = strided((b, tq, hq, d), kind, seed + 3, [0, 0, 0, pad], shift)
    before, base, outside = o.clone(), o._base, o._base.clone()
    lse = torch.full((b, hq, tq), 7.0, device="cuda") if with_lse else None
    scale = d ** -0.5 if scale is None else scale
    cross_attention(q, k, v, o, lse, None if q_lens is None else torch.tensor(ql, dtype=torch.int32, device="cuda"),
                    None if kv_lens is None else torch.tensor(kl, dtype=torch.int32, device="cuda"), given, scale, kind)
    done()
    ref, ref_lse, mag, dots = tokens.cross_attention(f64(q), f64(k), f64(v), ql, kl, mask, scale)
    got = f64(o)
    check_cross_result(got, lse, ref, ref_lse, mag, dots, kind, d, kv)
    o.copy_(before)  # nothing is written around the heads
    assert torch.equal(base.view(torch.int16), outside.view(torch.int16))
    return got


def check_cross_result(got, lse, ref, ref_lse, mag, dots, kind, d, kv):
    score = (d + 8) * 2.0 ** -23 * dots + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(ref_lse), ref_lse, 0)).max())
    # (weights relative to 2^7 of the largest, but for the 2^8 that it may stand above what they are relative to)
    tol = UNIT[kind] * np.abs(ref) + TINY[kind] + (2 * UNIT[kind] + 4 * score + 2.0 ** -18) * mag + TINY[kind] * 2 * kv * 8
    assert_within(got, ref, tol)
    fine = np.isfinite(ref_lse)
    assert (got[~fine.transpose(0, 2, 1)] == 0).all()
    if lse is not None:
        out = lse.double().cpu().numpy()
        assert np.array_equal(np.isneginf(out), np.isneginf(ref_lse))
        assert_within(out[fine], ref_lse[fine], np.full(fine.sum(), 2 * score + 2.0 ** -18))


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [8, 40, 64, 80, 128, 160, 256])
@pytest.mark.parametrize("tq,kv", [(1, 1), (1, 300), (3, 129), (40, 40), (130, 200), (300, 77), (600, 333)])
def test_cross_sizes(tq, kv, d, kind):
    check_cross(2, tq, kv, 4, 2, d, kind, seed=d)


@pytest.mark.parametrize("d", [1, 20, 63, 100, 129, 250])
@pytest.mark.parametrize("tq,kv", [(1, 70), (30, 70), (700, 150)])
def test_cross_odd_heads(tq, kv, d):
    check_cross(2, tq, kv, 2, 1, d, "fp16", seed=d)


@pytest.mark.parametrize("hq,hk", [(1, 1), (7, 1), (8, 8), (32, 4), (40, 1), (6, 2), (150, 1), (129, 1)])
@pytest.mark.parametrize("tq", [1, 2, 9, 90, 300])
def test_cross_shared_heads(tq, hq, hk):
    check_cross(2, tq, 150, hq, hk, 64, "fp16", seed=hq)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tq", [1, 4, 33, 160, 900])
def test_cross_ragged_lengths_and_empty_rows(tq, d):
    check_cross(7, tq, 200, 4, 2, d, "bf16", q_lens=[tq, tq, 0, max(1, tq // 2), tq, 1, tq],
                kv_lens=[200, 0, 50, 150, 64, 1, 129], seed=tq)


def masks(kv):
    rng = np.random.default_rng(kv)
    some = rng.random(kv) < 0.5
    return {"half": some, "first": np.arange(kv) < 1, "last": np.arange(kv) == kv - 1, "none": np.zeros(kv, bool),
            "all": np.ones(kv, bool), "late": np.arange(kv) >= min(kv - 1, 130), "holes": np.arange(kv) // 40 % 2 == 1}


@pytest.mark.parametrize("which", ["half", "first", "last", "none", "all", "late", "holes"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tq,kv", [(1, 300), (20, 65), (400, 300), (700, 77)])
def test_cross_masks(tq, kv, d, which):
    check_cross(3, tq, kv, 4, 4, d, "bf16", mask=masks(kv)[which], kv_lens=[kv, max(1, kv - 70), kv // 2], seed=kv)


@pytest.mark.parametrize("tq", [1, 350])
def test_cross_mask_of_each_sequence(tq):
    rng = np.random.default_rng(5)
    check_cross(6, tq, 190, 6, 2, 80, "fp16", mask=rng.random((6, 190)) < np.array([0, 0.02, 0.3, 0.9, 1, 0.5])[:, None],
                q_lens=[tq] * 5 + [tq // 2], seed=4)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("b,tq,kv,hq,hk", [(1, 1, 20000, 4, 1), (1, 300, 5000, 2, 2), (2, 1000, 4001, 2, 1), (1, 130, 9000, 1, 1),
                                           (1, 20, 6000, 8, 1), (1, 2500, 2000, 16, 16)])
def test_cross_long_keys(b, tq, kv, hq, hk, d):
    """Keys divided over clusters, over all SMs, and in many tiles."""
    check_cross(b, tq, kv, hq, hk, d, "bf16", kv_lens=[kv - 7, kv // 3][:b], seed=kv)


@pytest.mark.parametrize("d", [64, 128])
def test_cross_long_keys_with_a_mask_that_leaves_parts_empty(d):
    kv = 8000
    mask = (np.arange(kv) >= 5000) & (np.arange(kv) < 5100)
    for tq in (1, 300):
        check_cross(1, tq, kv, 2, 2, d, "fp16", mask=mask, seed=tq)


@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (3, 0), (0, 1), (8, 4)])
@pytest.mark.parametrize("tq", [1, 70, 600])
def test_cross_strides_and_alignment(tq, pad, shift):
    check_cross(2, tq, 140, 4, 2, 64, "bf16", pad=pad, shift=shift)


@pytest.mark.parametrize("tq", [1, 500])
@pytest.mark.parametrize("scale,size", [(1.0, 3.0), (0.0, 1.0), (-0.5, 1.0), (0.02, 12.0)])
def test_cross_sharp_and_flat_scores(tq, scale, size):
    check_cross(1, tq, 300, 2, 2, 64, "fp16", scale=scale, size=size, seed=3)


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [40, 64, 80, 128, 200])
@pytest.mark.parametrize("tq", [1, 300, 690])
def test_cross_scores_that_grow_along_the_keys(tq, d, kind):
    """Every 64 keys are larger than those before: sums and outputs are scaled again and again."""
    def edit(q, k, v):
        k *= (1 + torch.arange(700, device="cuda") // 64 * 2).to(k.dtype)[None, :, None, None]

    check_cross(1, tq, 700, 4, 2, d, kind, edit=edit, seed=d + tq)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_cross_many_items_a_cta(d):
    """More row tiles than the device holds at once, of sequences of all lengths."""
    rng = np.random.default_rng(d)
    b = 12
    check_cross(b, 700, 190, 8, 8, d, "bf16", q_lens=rng.integers(0, 701, b), kv_lens=rng.integers(0, 191, b), seed=d)


def test_cross_many_sequences_of_single_tokens():
    rng = np.random.default_rng(4)
    check_cross(90, 1, 260, 8, 2, 128, "bf16", kv_lens=rng.integers(0, 261, 90), seed=6)


@pytest.mark.parametrize("tq", [1, 400])
def test_cross_numbers_that_are_none_reach_the_rows_that_see_them(tq):
    q, k, v = (strided((2, n, 2, 64), "bf16", n) for n in (tq, 200, 200))
    v[0, 50, 0, 5] = float("inf")
    k[1, 60, 1, 3] = float("nan")
    o = torch.zeros_like(q)
    cross_attention(q, k, v, o, None, None, None, None, 0.125, "bf16")
    done()
    bad = torch.zeros_like(o, dtype=torch.bool)
    bad[0, :, 0, 5], bad[1, :, 1] = True, True
    assert torch.equal(~o.isfinite(), bad)


@pytest.mark.parametrize("tq", [1, 600])
def test_cross_shared_operands_and_strides_of_single_elements(tq):
    """Queries shared by sequences, keys and values by sequences and heads; strides that mean nothing."""
    q = strided((1, tq, 4, 64), "bf16", 1).expand(3, tq, 4, 64)
    k, v = (strided((1, 200, 1, 64), "bf16", i).expand(3, 200, 2, 64) for i in (2, 3))
    mask = (torch.arange(200, device="cuda") % 3 > 0).to(torch.uint8)[None].expand(3, 200)
    o, lse = torch.empty(3, tq, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 4, tq, device="cuda")
    cross_attention(q, k, v, o, lse, None, None, mask, 0.125, "bf16")
    done()
    ref = tokens.cross_attention(f64(q), f64(k), f64(v), [tq] * 3, [200] * 3, mask.cpu().numpy(), 0.125)
    check_cross_result(f64(o), lse, *ref, "bf16", 64, 200)
    import conv2d_implicit_gemm_gb300 as ox
    q1, k1, v1 = q[:1, :, :1].contiguous(), k[:1, :, :1].contiguous(), v[:1, :, :1].contiguous()
    o1 = torch.zeros(1, tq, 1, 64, dtype=torch.bfloat16, device="cuda")
    ox.oidnx_cross_attention(q1.data_ptr(), 3, q1.stride(1), 5, k1.data_ptr(), 0, k1.stride(1), 1, v1.data_ptr(), -7,
                             v1.stride(1), 9, o1.data_ptr(), 11, o1.stride(1), 13, 0, 0, 0, mask.data_ptr(), 0, 1, tq, 200, 1,
                             1, 64, 0.125, ox.PRECISION_BF16, torch.cuda.current_stream().cuda_stream)
    done()
    assert_within(f64(o1), ref[0][:1, :, :1], (UNIT["bf16"] * np.abs(ref[0]) + (2 * UNIT["bf16"] + 2.0 ** -14) * ref[2])[:1, :, :1])


def test_cross_heads_before_tokens():
    """Heads outside, tokens inside ([b][h][t][d] in memory), and outputs the other way round."""
    q, k, v = (strided((2, 4, n, 80), "fp16", n).transpose(1, 2) for n in (500, 150, 150))
    o, lse = torch.empty(2, 500, 4, 80, dtype=torch.float16, device="cuda"), torch.empty(2, 4, 500, device="cuda")
    cross_attention(q, k, v, o, lse, None, None, None, 0.1, "fp16")
    done()
    ref = tokens.cross_attention(f64(q), f64(k), f64(v), [500] * 2, [150] * 2, None, 0.1)
    check_cross_result(f64(o), lse, *ref, "fp16", 80, 150)


def test_cross_without_keys_is_zero():
    q = strided((2, 300, 4, 64), "fp16", 1)
    o, lse = torch.ones_like(q), torch.ones(2, 4, 300, device="cuda")
    cross_attention(q, q[:, :0], q[:, :0], o, lse, None, None, None, 0.125, "fp16")
    done()
    assert not o.any() and lse.isneginf().all()


def test_cross_keys_beyond_32_bit_offsets():
    kv, hk, d = 2 ** 31 // 512 + 4096, 4, 128
    k = torch.zeros(1, kv, hk, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    tail = strided((1, 300, hk, d), "bf16", 1)
    k[:, -300:], v[:, -300:] = tail, tail.flip(1)
    mask = torch.zeros(1, kv, dtype=torch.uint8, device="cuda")
    mask[:, -300:] = 1
    for tq in (1, 150):
        q = strided((1, tq, hk, d), "bf16", 2)
        o, lse = torch.empty_like(q), torch.empty(1, hk, tq, device="cuda")
        cross_attention(q, k, v, o, lse, None, None, mask, d ** -0.5, "bf16")
        done()
        ref = tokens.cross_attention(f64(q), f64(k[:, -300:]), f64(v[:, -300:]), [tq], [300], None, d ** -0.5)
        check_cross_result(f64(o), lse, *ref, "bf16", d, 300)


@pytest.mark.parametrize("tq", [1, 300])
def test_cross_repeated_tokens_and_heads(tq):
    """Strides of 0 and below it that no tensor map takes: one query for all tokens and heads, keys in reverse, one value."""
    q = strided((2, 1, 1, 64), "fp16", 1).expand(2, tq, 4, 64)
    back = strided((2, 90, 2, 64), "fp16", 2)
    v = strided((2, 1, 2, 64), "fp16", 3).expand(2, 90, 2, 64)
    o, lse = torch.empty(2, tq, 4, 64, dtype=torch.float16, device="cuda"), torch.empty(2, 4, tq, device="cuda")
    import conv2d_implicit_gemm_gb300 as ox
    ox.oidnx_cross_attention(q.data_ptr(), *q.stride()[:3], back[:, -1].data_ptr(), back.stride(0), -back.stride(1),
                             back.stride(2), v.data_ptr(), *v.stride()[:3], o.data_ptr(), *o.stride()[:3], lse.data_ptr(), 0, 0,
                             0, 0, 2, tq, 90, 4, 2, 64, 0.125, ox.PRECISION_FP16, torch.cuda.current_stream().cuda_stream)
    done()
    ref = tokens.cross_attention(f64(q), f64(back.flip(1)), f64(v), [tq] * 2, [90] * 2, None, 0.125)
    check_cross_result(f64(o), lse, *ref, "fp16", 64, 90)


# ---------------------------------------------------------------- all of them
def example_of(name):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", name + ".py")
    spec = importlib.util.spec_from_file_location(name, path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("sizes", [dict(), dict(channels=384, heads=6, key_heads=2, head=80, text=200, length=130),
                                   dict(batch=3, shape=(1, 7, 9), length=1)])
def test_a_block_of_them_follows_its_definition(sizes, dtype):
    """The example's block against 64 bits: twelve roundings to 16 bits lie on the way of the last norm, none of whose
    relative errors (half a unit at most) a norm, an average or a projection of random weights enlarges beyond its factor
    of at most 2 (scale, gate and weights together)."""
    total, normed = example_of("video_block").run(dtype=dtype, **sizes)
    unit = UNIT["fp16" if dtype == torch.float16 else "bf16"]
    assert total <= 24 * unit and normed <= 24 * unit


def calls_of_every_form():
    """One call of each form, each writing the returned tensors."""
    out = []

    def cross(b, tq, kv, hq, hk, d, pad=0, mask=False):
        q, k, v = strided((b, tq, hq, d), "bf16", tq, [0, 0, 0, pad]), strided((b, kv, hk, d), "bf16", kv), strided((b, kv, hk, d), "bf16", 3)
        o, lse = strided((b, tq, hq, d), "bf16", 4, [0, 0, 0, pad]), torch.empty(b, hq, tq, device="cuda")
        seen = (torch.arange(kv, device="cuda") % 5 > 0).to(torch.uint8)[None].repeat(b, 1) if mask else None
        out.append((lambda: cross_attention(q, k, v, o, lse, None, None, seen, d ** -0.5, "bf16"), (o, lse)))

    cross(2, 1, 300, 4, 2, 64)              # few queries
    cross(1, 1, 3000, 4, 4, 128)            # divided over a cluster
    cross(1, 1, 30000, 2, 1, 128)           # over many CTAs, with a kernel that joins them
    cross(3, 700, 333, 6, 2, 80, mask=True) # tiles
    cross(1, 300, 5000, 2, 2, 64)           # tiles divided over a cluster
    cross(2, 200, 150, 4, 4, 60, pad=1)     # copied first
    for t, n in ((3, 500), (3, 501), (900, 1024), (900, 1001), (400, 17000)):
        x, w = strided((t, n), "bf16", t), strided((n,), "bf16", n)
        r, s, y = strided((t, n), "fp32", 2), torch.empty(t, n, device="cuda"), torch.empty(t, n, dtype=torch.bfloat16, device="cuda")
        out.append((lambda x=x, r=r, s=s, y=y, w=w, t=t: block_norm(x, r, s, y, "rms", w, None, "layer", w, w, 1e-6, None, "plain",
                                                               None, None, None, t, 1, 1.0, 0.5, "bf16", "fp32"), (s, y)))
    for d in (128, 66):
        q, k, v = (strided((50, h, d), "bf16", h) for h in (4, 2, 2))
        got = [torch.empty_like(z) for z in (q, k, v)]
        table = torch.randn(60, 24, device="cuda")
        at = torch.arange(150, dtype=torch.int32, device="cuda").view(3, 50) % 60
        out.append((lambda q=q, k=k, v=v, got=got, table=table, at=at: norm_rope_axes(
            q, got[0], k, got[1], v, got[2], True, None, None, 1e-6, table, table, at, [r % 3 for r in range(24)], None, False, "bf16"), got))
    return out


def test_block_calls_captured_and_replayed_on_two_streams_at_once():
    """Two graphs of every form, each with its own outputs, replayed at the same time, give what the calls gave."""
    sets = [calls_of_every_form() for _ in range(2)]
    graphs, refs = [], []
    for calls in sets:
        for call, _ in calls:
            call()
        done()
        refs.append([t.clone() for _, outs in calls for t in outs])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for call, _ in calls:
                call()
        graphs.append(g)
        for _, outs in calls:
            for t in outs:
                t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for calls, ref in zip(sets, refs):
        assert all(torch.equal(a, b) for a, b in zip([t for _, outs in calls for t in outs], ref))


def test_block_results_do_not_depend_on_the_stream_or_on_what_ran_before():
    calls = calls_of_every_form()
    loud = [strided((2, 300, 4, d), "fp16", 4, scale=30.0) for d in (64, 128, 256)]
    first = None
    side = torch.cuda.Stream()
    for s in (torch.cuda.current_stream(), side, side, torch.cuda.current_stream()):
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            for x in loud:
                cross_attention(x, x, x, torch.empty_like(x), None, None, None, None, 1.0, "fp16")
            for call, _ in calls:
                call()
            done()
            got = [t.clone() for _, outs in calls for t in outs]
        torch.cuda.synchronize()
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_block_calls_from_a_thread_of_its_own():
    import threading
    calls = calls_of_every_form()
    for call, _ in calls:
        call()
    done()
    ref = [t.clone() for _, outs in calls for t in outs]
    failed = []

    def work():
        try:
            for call, _ in calls:
                call()
            done()
        except Exception as e:
            failed.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed
    assert all(torch.equal(a, b) for a, b in zip([t for _, outs in calls for t in outs], ref))


# ---------------------------------------------------------------- what the calls take besides
@pytest.mark.parametrize("tq", [1, 300])
def test_cross_lengths_outside_the_buffers(tq):
    """More keys or queries than there is room for are read as what there is; fewer than none as none."""
    q, k, v = strided((4, tq, 2, 64), "bf16", 1), strided((4, 100, 2, 64), "bf16", 2), strided((4, 100, 2, 64), "bf16", 3)
    ql, kl = [tq + 5, tq, -3, 2 ** 31 - 1], [101, -1, 50, 2 ** 31 - 1]
    o, lse = torch.full_like(q, 9), torch.full((4, 2, tq), 9.0, device="cuda")
    cross_attention(q, k, v, o, lse, torch.tensor(ql, dtype=torch.int32, device="cuda"),
                    torch.tensor(kl, dtype=torch.int32, device="cuda"), None, 0.125, "bf16")
    done()
    ref = tokens.cross_attention(f64(q), f64(k), f64(v), [tq, tq, 0, tq], [100, 0, 50, 100], None, 0.125)
    check_cross_result(f64(o), lse, *ref, "bf16", 64, 100)


@pytest.mark.parametrize("d", [64, 128])
def test_cross_one_mask_row_and_no_statistics(d):
    """A mask shared by all sequences through a stride of 0, lse left out."""
    q, k, v = strided((3, 200, 4, d), "fp16", 1), strided((3, 140, 4, d), "fp16", 2), strided((3, 140, 4, d), "fp16", 3)
    mask = (torch.arange(140, device="cuda") % 7 > 2).to(torch.uint8)
    o = torch.zeros_like(q)
    cross_attention(q, k, v, o, None, None, None, mask[None].expand(3, 140), d ** -0.5, "fp16")
    done()
    ref = tokens.cross_attention(f64(q), f64(k), f64(v), [200] * 3, [140] * 3, np.broadcast_to(mask.cpu().numpy(), (3, 140)), d ** -0.5)
    check_cross_result(f64(o), None, *ref, "fp16", d, 140)


def test_cross_more_heads_a_key_head_than_a_row_tile_has_rows():
    check_cross(1, 70, 333, 200, 1, 128, "bf16", seed=2)


@pytest.mark.parametrize("tq", [1, 200])
def test_cross_queries_of_a_fused_projection(tq):
    """Queries, keys and values as one projection wrote them, in one buffer."""
    qkv = strided((2, tq, 12, 64), "bf16", 1)
    q, k, v = qkv[:, :, :8], qkv[:, :, 8:10], qkv[:, :, 10:]
    o, lse = torch.empty(2, tq, 8, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 8, tq, device="cuda")
    cross_attention(q, k, v, o, lse, None, None, None, 0.125, "bf16")
    done()
    ref = tokens.cross_attention(f64(q), f64(k), f64(v), [tq] * 2, [tq] * 2, None, 0.125)
    check_cross_result(f64(o), lse, *ref, "bf16", 64, tq)


@pytest.mark.parametrize("t,n", [(5, 320), (1000, 321)])
def test_block_norm_groups_without_a_count_of_rows(t, n):
    """Rows named by groups need no per; the same group may come back."""
    rng = np.random.default_rng(t)
    check_block(t, n, "fp16", per=0, count=4, groups=np.sort(rng.integers(0, 4, t))[rng.permutation(t)])


def test_block_norm_small_values_and_no_eps():
    """Values whose squares are far below 1, and eps = 0."""
    x = strided((400, 512), "bf16", 1, scale=1e-12)
    y = torch.empty_like(x)
    block_norm(x, None, None, y, "none", None, None, "layer", None, None, 0.0, None, "plain", None, None, None, 400, 1, 1.0, 1.0,
               "bf16", "bf16")
    done()
    _, ref, _, size = tokens.block_norm(f64(x), None, "none", None, None, "layer", None, None, 0.0, None, "plain", None, None, 1.0, 1.0)
    assert_within(f64(y), ref, UNIT["bf16"] * np.abs(ref) + 96 * 2.0 ** -24 * size)
