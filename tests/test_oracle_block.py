"""Pins of the 64-bit definitions of a conditioned block's operators: torch CPU float64 library routines, complex
rotations, sums written out."""

import numpy as np
import pytest
import torch
import torch.nn.functional as F

from oracle import tokens


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("act", ["plain", "tanh", "sigmoid"])
def test_block_norm_matches_torch(post, pre, act):
    rng = np.random.default_rng(len(post) + 3 * len(pre) + len(act))
    t, n = 4, 9
    x, r, gate, scale, shift = (rng.standard_normal((t, n)) * 2 + 0.5 for _ in range(5))
    w, b, u, c = (rng.standard_normal(n) for _ in range(4))

    def norm(z, kind, weight, bias):
        if kind == "none":
            return z
        weight, bias = torch.from_numpy(weight), torch.from_numpy(bias)
        return F.layer_norm(z, (n,), weight, bias, 1e-3) if kind == "layer" else F.rms_norm(z, (n,), weight, 1e-3) + bias

    g = {"plain": lambda z: z, "tanh": torch.tanh, "sigmoid": torch.sigmoid}[act](torch.from_numpy(gate))
    total = 0.75 * torch.from_numpy(r) - 1.5 * g * norm(torch.from_numpy(x), post, w, b)
    y = norm(total, pre, u, c) * (1 + torch.from_numpy(scale)) + torch.from_numpy(shift)
    got = tokens.block_norm(x, r, post, w, b, pre, u, c, 1e-3, gate, act, scale, shift, 0.75, -1.5)
    assert np.allclose(got[0], total.numpy(), rtol=1e-12, atol=1e-12) and np.allclose(got[1], y.numpy(), rtol=1e-12, atol=1e-12)
    assert (np.abs(got[0]) <= got[2] + 1e-12).all() and (np.abs(got[1]) <= got[3] + 1e-12).all()


def test_block_norm_magnitudes_bound_what_an_error_does():
    """A relative change of every value moves the results by no more than twice that of their magnitudes."""
    rng = np.random.default_rng(1)
    x, r = rng.standard_normal((3, 40)) + 3, rng.standard_normal((3, 40)) + 2
    for kind in ("rms", "layer"):
        call = lambda a, b: tokens.block_norm(a, b, kind, None, None, kind, None, None, 1e-6, None, "plain", None, None, 1.0, 1.0)  # noqa: E731
        ref = call(x, r)
        step = 1e-7
        got = call(x * (1 + step * rng.uniform(-1, 1, x.shape)), r * (1 + step * rng.uniform(-1, 1, x.shape)))
        assert (np.abs(got[0] - ref[0]) <= 2 * step * ref[2]).all() and (np.abs(got[1] - ref[1]) <= 2 * step * ref[3]).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_axes_are_complex_rotations_by_their_own_positions(interleaved):
    rng = np.random.default_rng(3)
    axes, pairs = [0, 2, 1, 2, 0], 5
    table = rng.uniform(-3, 3, (7, pairs))
    at = rng.integers(0, 7, (3, 6))
    x = rng.standard_normal((6, 2, 12))
    cos, sin = tokens.axes_rows(np.cos(table), at, axes), tokens.axes_rows(np.sin(table), at, axes)
    got, _ = tokens.norm_rope(x, None, 0.0, cos, sin, 2 * pairs, interleaved, norm=False)
    for i in range(6):
        for r, axis in enumerate(axes):
            a, b = (2 * r, 2 * r + 1) if interleaved else (r, r + pairs)
            z = (x[i, :, a] + 1j * x[i, :, b]) * np.exp(1j * table[at[axis, i], r])
            assert np.allclose(got[i, :, a], z.real) and np.allclose(got[i, :, b], z.imag)
    assert np.array_equal(got[..., 10:], x[..., 10:])


def test_axes_outside_the_table_are_nan():
    out = tokens.axes_rows(np.ones((4, 3)), np.array([[0, -1], [4, 3]]), [0, 1, 0])
    assert np.array_equal(np.isnan(out), [[False, True, False], [True, False, True]])


@pytest.mark.parametrize("group", [1, 3])
def test_cross_attention_matches_torch(group):
    rng = np.random.default_rng(group)
    b, tq, kv, hk, d = 3, 5, 7, 2, 4
    q, k, v = rng.standard_normal((b, tq, hk * group, d)), rng.standard_normal((b, kv, hk, d)), rng.standard_normal((b, kv, hk, d))
    lens, mask = np.array([7, 4, 0]), rng.random((b, kv)) < 0.7
    mask[:, 0] = True
    o, lse, size, dots = tokens.cross_attention(q, k, v, [5, 3, 5], lens, mask, 0.6)
    for s in range(b):
        seen = (np.arange(kv) < lens[s]) & mask[s]
        n = (5, 3, 5)[s]
        if not seen.any():
            assert not o[s].any() and np.isneginf(lse[s]).all()
            continue
        kk, vv = (torch.from_numpy(z[s]).repeat_interleave(group, 1).transpose(0, 1) for z in (k, v))
        ref = F.scaled_dot_product_attention(torch.from_numpy(q[s]).transpose(0, 1), kk, vv, torch.from_numpy(seen)[None, None].expand(1, tq, kv), scale=0.6)
        assert np.allclose(o[s, :n], ref.transpose(0, 1).numpy()[:n])
        assert not o[s, n:].any() and np.isneginf(lse[s, :, n:]).all()
        score = np.einsum("ihd,jhd->hij", q[s, :n], np.repeat(k[s], group, 1)) * 0.6
        assert np.allclose(lse[s, :, :n], np.log(np.exp(score[:, :, seen]).sum(-1)))
        assert (np.abs(o[s]) <= size[s] + 1e-12).all() and np.abs(score[:, :, seen]).max() <= dots + 1e-12
