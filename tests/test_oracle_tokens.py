"""Pins of the token operators' 64-bit definitions: torch CPU float64 library routines, complex rotations, caches written
key by key, closed forms."""

import math

import numpy as np
import pytest
import torch
import torch.nn.functional as F

from oracle import tokens

ACTS = {"none": lambda z: z, "relu": F.relu, "gelu": F.gelu, "gelu_tanh": lambda z: F.gelu(z, approximate="tanh"),
        "silu": F.silu}


# ---------------------------------------------------------------- linear
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("seed", range(4))
def test_linear_matches_torch(act, seed):
    rng = np.random.default_rng(seed)
    m, n, k = rng.integers(1, 12, 3)
    x, w, b, r = (rng.standard_normal(s) * 2 for s in ((m, k), (n, k), (n,), (m, n)))
    ref = ACTS[act](F.linear(torch.from_numpy(x), torch.from_numpy(w), torch.from_numpy(b))).numpy()
    got, size = tokens.linear(x, w, b, r, act)
    assert np.allclose(got, ref + r, rtol=1e-12, atol=1e-12)
    assert np.allclose(tokens.linear(x, w, b, None, act)[0], ref, rtol=1e-12, atol=1e-12)
    # the magnitudes bound every partial sum
    sums = np.cumsum(x[:, None, :] * w[None], axis=-1) + b[None, :, None]
    assert (np.abs(sums) <= size[..., None] + 1e-12).all()


@pytest.mark.parametrize("act", ACTS)
def test_activations_over_their_range(act):
    z = np.concatenate([np.linspace(-30, 30, 2001), [0.0, -0.0, 1e-30, -1e-30, 1e4, -1e4, 1e30]])
    ref = ACTS[act](torch.from_numpy(z)).numpy()
    # the definitions with 1 + erf and 1 + tanh lose what they cancel: relative to |z|
    assert (np.abs(tokens.activation(z, act) - ref) <= 1e-15 * np.abs(z) + 1e-15 * np.abs(ref)).all()


@pytest.mark.parametrize("act,low", [("none", -np.inf), ("relu", 0.0), ("gelu", np.nan), ("gelu_tanh", np.nan), ("silu", np.nan)])
def test_activations_at_infinity(act, low):
    """The limits above; below, 0 x infinity where the formula says so."""
    with np.errstate(invalid="ignore", over="ignore"):
        got = tokens.activation(np.array([np.inf, -np.inf, np.nan]), act)
    assert np.isposinf(got[0]) and np.isnan(got[2])
    np.testing.assert_array_equal(got[1], low)


def test_linear_without_products():
    got, size = tokens.linear(np.zeros((2, 0)), np.zeros((3, 0)), np.array([-1.0, 0.0, 2.0]), np.ones((2, 3)), "relu")
    assert np.array_equal(got, [[1, 1, 3]] * 2) and np.array_equal(size, [[1, 0, 2]] * 2)


# ---------------------------------------------------------------- norm and rotation
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(2, 2), (8, 8), (10, 4), (7, 0), (9, 6)])
def test_norm_rope_is_a_complex_rotation(d, rot, interleaved):
    rng = np.random.default_rng(d)
    x, w = rng.standard_normal((5, 3, d)), rng.standard_normal(d)
    angle = rng.uniform(-4, 4, (5, rot // 2))
    got, size = tokens.norm_rope(x, w, 1e-3, np.cos(angle), np.sin(angle), rot, interleaved)
    y = x / np.sqrt(np.square(x).sum(-1, keepdims=True) / d + 1e-3) * w
    first = y[..., 0:rot:2] if interleaved else y[..., :rot // 2]
    second = y[..., 1:rot:2] if interleaved else y[..., rot // 2:rot]
    z = (first + 1j * second) * np.exp(1j * angle)[:, None]
    turned = np.stack([z.real, z.imag], -1 if interleaved else -2).reshape(5, 3, rot)
    assert np.allclose(got, np.concatenate([turned, y[..., rot:]], -1), rtol=1e-12, atol=1e-13)
    assert (np.abs(got) <= size + 1e-12).all()


def test_norm_has_unit_mean_square_and_depends_on_distance_only():
    """Without eps and weight heads have mean square 1, and a product of two rotated heads depends on the difference of
    their positions."""
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))
    freq = 10.0 ** -np.arange(8)

    def at(x, p):
        return tokens.norm_rope(x, None, 0.0, np.cos(p * freq)[None], np.sin(p * freq)[None], 16, False)[0][0, 0]

    assert abs(np.square(at(q, 5)).mean() - 1) < 1e-12
    assert abs(at(q, 9) @ at(k, 2) - at(q, 107) @ at(k, 100)) < 1e-10


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("cap,sinks", [(1, 0), (5, 0), (5, 2), (5, 4), (5, 5), (5, 9), (8, 3)])
def test_held_positions_are_what_sequential_writes_leave(cap, sinks):
    """Keys written one after the other: into free slots first, then round the slots behind the sinks."""
    slots, ring = {}, min(sinks, cap)
    at = ring
    for n in range(40):
        assert tokens.held_positions(n, cap, sinks) == {j: s for s, j in slots.items()}
        if n < cap:
            slots[n] = n
        elif ring < cap:
            slots[at] = n
            at = at + 1 if at + 1 < cap else ring


def _masked(q, k, v, mask, scale):
    """torch's attention in 64 bits over [heads][rows][d] with a mask of what is seen."""
    group = q.shape[1] // k.shape[1]
    t = [torch.from_numpy(np.ascontiguousarray(a.transpose(1, 0, 2))) for a in (q, k, v)]
    t[1], t[2] = (a.repeat_interleave(group, 0) for a in t[1:])
    o = F.scaled_dot_product_attention(*t, attn_mask=torch.from_numpy(mask), scale=scale)
    z = (t[0] @ t[1].transpose(1, 2) * scale).masked_fill(~torch.from_numpy(mask), -math.inf)
    return o.numpy().transpose(1, 0, 2), torch.logsumexp(z, -1).numpy()


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (3, 2), (50, 0), (2, 9)])
@pytest.mark.parametrize("tq,kv,hq,hk", [(1, 9, 2, 2), (4, 9, 4, 2), (9, 9, 3, 1)])
def test_window_attention_matches_torch_over_a_linear_cache(tq, kv, hq, hk, window, sinks):
    rng = np.random.default_rng(tq)
    q, k, v = rng.standard_normal((1, tq, hq, 6)), rng.standard_normal((1, 12, hk, 6)), rng.standard_normal((1, 12, hk, 6))
    p, j = kv - tq + np.arange(tq)[:, None], np.arange(kv)[None]
    mask = (j <= p) & ((window == 0) | (j > p - window) | (j < sinks))
    ref, ref_lse = _masked(q[0], k[0, :kv], v[0, :kv], mask, 0.3)
    o, lse, size, dots = tokens.window_attention(q, k, v, [tq], [kv], window, sinks, 0.3)
    assert np.allclose(o[0], ref, rtol=1e-12, atol=1e-13) and np.allclose(lse[0], ref_lse, rtol=1e-12, atol=1e-13)
    assert (np.abs(o) <= size + 1e-12).all()
    assert dots >= np.abs(np.einsum("qhd,khd->qkh", q[0], np.repeat(k[0, :kv], hq // hk, 1))[mask]).max() * 0.3 - 1e-12


@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 1), (0, 2), (4, 0)])
@pytest.mark.parametrize("tq,cap,kv", [(1, 6, 17), (3, 6, 17), (9, 5, 9), (6, 6, 30)])
def test_window_attention_over_a_ring_is_attention_over_the_keys_that_stay(tq, cap, kv, window, sinks):
    """Prompts longer than the ring among them: rows whose keys are all gone are 0 with lse -inf."""
    rng = np.random.default_rng(kv)
    q, keys, values = rng.standard_normal((1, tq, 2, 4)), rng.standard_normal((kv, 1, 4)), rng.standard_normal((kv, 1, 4))
    k, v = np.full((1, cap, 1, 4), np.nan), np.full((1, cap, 1, 4), np.nan)
    stays, at = {}, sinks
    for n in range(kv):
        slot = n if n < cap else at
        if n >= cap:
            at = at + 1 if at + 1 < cap else sinks
        k[0, slot], v[0, slot], stays[slot] = keys[n], values[n], n
    held = np.isin(np.arange(kv), list(stays.values()))[None]
    p, j = kv - tq + np.arange(tq)[:, None], np.arange(kv)[None]
    mask = held & (j <= p) & ((window == 0) | (j > p - window) | (j < sinks))
    o, lse, *_ = tokens.window_attention(q, k, v, [tq], [kv], window, sinks, 1.0)
    some = mask.any(1)
    ref, ref_lse = _masked(q[0][some], keys, values, mask[some], 1.0)
    assert np.allclose(o[0][some], ref, rtol=1e-12, atol=1e-13) and np.allclose(lse[0][:, some], ref_lse, rtol=1e-12)
    assert not o[0][~some].any() and np.isneginf(lse[0][:, ~some]).all()


def test_window_attention_lengths():
    """Rows from q_len on, rows before the first key and sequences without keys are empty; others do not see each other."""
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((4, 3, 1, 4)), rng.standard_normal((4, 5, 1, 4)), rng.standard_normal((4, 5, 1, 4))
    o, lse, *_ = tokens.window_attention(q, k, v, [2, 3, 3, 0], [5, 0, 1, 5], 0, 0, 1.0)
    empty = np.array([[0, 0, 1], [1, 1, 1], [1, 1, 0], [1, 1, 1]], bool)
    assert not o[empty].any() and np.isneginf(lse[:, 0][empty]).all() and np.isfinite(lse[:, 0][~empty]).all()
    assert np.allclose(o[2, 2], v[2, 0])  # one key: its value
    alone = tokens.window_attention(q[:1], k[:1], v[:1], [2], [5], 0, 0, 1.0)[0]
    assert np.array_equal(alone[0], o[0])
