"""The token operators in 64 bits, from their definitions: the linear layer with
its epilogue, the norm and rotation of heads, attention with a sliding window and
sinks over a linear or ring cache, the norms around a branch, and attention to an
encoder's states.  numpy float64, no tricks; each also returns the magnitudes that
its rounding errors scale with."""

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])


def activation(z, act):
    if act == "relu":
        return np.where(z < 0, 0.0, z)
    if act == "gelu":
        return 0.5 * z * (1 + _erf(z / math.sqrt(2))) if z.size else z
    if act == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        with np.errstate(over="ignore"):
            return z / (1 + np.exp(-z))
    return z


def linear(x, w, bias=None, residual=None, act="none"):
    """(y, magnitude of the sums before the activation)."""
    z = x @ w.T
    size = np.abs(x) @ np.abs(w).T
    if bias is not None:
        z, size = z + bias, size + np.abs(bias)
    y = activation(z, act)
    return (y if residual is None else y + residual), size


def norm_rope(x, weight, eps, cos, sin, rot, interleaved, norm=True):
    """x [t][h][d], cos and sin [t][rot / 2]: (y, magnitude |a| + |b| per value)."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) if norm else x
    if weight is not None:
        y = y * weight
    out, size = y.copy(), np.abs(y)
    for r in range(rot // 2):
        i, j = (2 * r, 2 * r + 1) if interleaved else (r, r + rot // 2)
        a, b = y[..., i], y[..., j]
        c, s = cos[:, None, r], sin[:, None, r]
        out[..., i], out[..., j] = a * c - b * s, b * c + a * s
        size[..., i] = size[..., j] = np.abs(a) + np.abs(b)
    return out, size


def axes_rows(table, positions, pair_axes):
    """table [rows][pairs] at row positions[pair_axes[r]][i] for pair r of token i (NaN outside it): [t][pairs]."""
    out = np.full((positions.shape[1], len(pair_axes)), np.nan)
    for r, axis in enumerate(pair_axes):
        at = positions[axis]
        known = (at >= 0) & (at < table.shape[0])
        out[known, r] = table[at[known], r]
    return out


def _norm(z, size, kind, weight, bias, eps):
    """(normed z, the magnitude that its errors scale with), where z is off by multiples of `size`."""
    if kind == "none":
        return z, size
    mean = z.mean(-1, keepdims=True) if kind == "layer" else 0.0
    size = size + (size.mean(-1, keepdims=True) if kind == "layer" else 0.0)
    c = z - mean
    root = 1 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    w = np.abs(weight) if weight is not None else 1.0
    # the root is off by what the rows' deviations are off by, relative to their own size
    size = w * root * (size + np.abs(c) * (1 + root * np.sqrt((size * size).mean(-1, keepdims=True))))
    y = c * root
    y = y if weight is None else y * weight
    return (y, size) if bias is None else (y + bias, size + np.abs(bias))


def block_norm(x, residual, post, post_weight, post_bias, pre, pre_weight, pre_bias, eps, gate, gate_act, scale, shift,
               residual_scale, branch_scale):
    """x [t][n], gate, scale and shift [t][n] or None: (sum, y, the magnitudes of both)."""
    z, size = _norm(x, np.abs(x), post, post_weight, post_bias, eps)
    if gate is not None:
        g = {"plain": lambda v: v, "tanh": np.tanh, "sigmoid": lambda v: 1 / (1 + np.exp(-v))}[gate_act](gate)
        z, size = z * g, size * np.abs(g)
    z, size = z * branch_scale, size * abs(branch_scale)
    if residual is not None:
        z, size = z + residual_scale * residual, size + np.abs(residual_scale * residual)
    y, size_y = _norm(z, size, pre, pre_weight, pre_bias, eps)
    if scale is not None:
        y, size_y = y * (1 + scale), size_y * (1 + np.abs(scale))
    if shift is not None:
        y, size_y = y + shift, size_y + np.abs(shift)
    return z, y, size, size_y


def held_positions(n, cap, sinks):
    """{position: slot} of the keys that a cache of cap slots holds after n writes."""
    held = {}
    for j in range(n):
        if j < cap:
            slot = j
        elif sinks < cap:
            slot = sinks + (j - sinks) % (cap - sinks)
        else:
            continue
        held[slot] = j
    return {j: slot for slot, j in held.items()}


def window_attention(q, k, v, q_lens, kv_lens, window, sinks, scale):
    """q [b][tq][hq][d], k and v [b][cap][hk][d]: (o, lse, sum p |v|, largest sum |q||k|)."""
    b, tq, hq, d = q.shape
    cap, hk = k.shape[1:3]
    o = np.zeros_like(q)
    size = np.zeros_like(q)
    lse = np.full((b, hq, tq), -np.inf)
    dots = 0.0
    for s in range(b):
        held = held_positions(int(kv_lens[s]), cap, sinks)
        at = np.array(sorted(held), np.int64)
        slots = np.array([held[j] for j in sorted(held)], np.int64)
        for i in range(int(q_lens[s])):
            p = int(kv_lens[s]) - int(q_lens[s]) + i
            seen = at <= p
            if window:
                seen &= (at > p - window) | (at < sinks)
            use = slots[seen]
            if not len(use):
                continue
            for h in range(hq):
                kk, vv = k[s, use, h // (hq // hk)], v[s, use, h // (hq // hk)]
                z = kk @ q[s, i, h] * scale
                top = z.max()
                e = np.exp(z - top)
                lse[s, h, i] = top + math.log(e.sum())
                w = e / e.sum()
                o[s, i, h] = w @ vv
                size[s, i, h] = w @ np.abs(vv)
                dots = max(dots, float((np.abs(kk) @ np.abs(q[s, i, h])).max()) * abs(scale))
    return o, lse, size, dots


def cross_attention(q, k, v, q_lens, kv_lens, mask, scale):
    """q [b][tq][hq][d], k and v [b][kv][hk][d], mask [b][kv] or None: (o, lse, sum p |v|, largest sum |q||k|)."""
    b, tq, hq, d = q.shape
    kv, hk = k.shape[1:3]
    o, size = np.zeros_like(q), np.zeros_like(q)
    lse = np.full((b, hq, tq), -np.inf)
    dots = 0.0
    for s in range(b):
        use = np.arange(kv) < kv_lens[s]
        if mask is not None:
            use &= mask[s] != 0
        nq = int(q_lens[s])
        if not use.any() or nq == 0:
            continue
        for h in range(hq):
            kk, vv, qq = k[s, use, h // (hq // hk)], v[s, use, h // (hq // hk)], q[s, :nq, h]
            z = qq @ kk.T * scale
            top = z.max(-1, keepdims=True)
            e = np.exp(z - top)
            total = e.sum(-1, keepdims=True)
            lse[s, h, :nq] = (top + np.log(total))[:, 0]
            o[s, :nq, h] = e / total @ vv
            size[s, :nq, h] = e / total @ np.abs(vv)
            dots = max(dots, float((np.abs(qq) @ np.abs(kk).T).max()) * abs(scale))
    return o, lse, size, dots
