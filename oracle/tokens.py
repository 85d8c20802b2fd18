"""The token operators in 64 bits, from their definitions: the linear layer with
its epilogue, the norm and rotation of heads, and attention with a sliding
window and sinks over a linear or ring cache.  numpy float64, no tricks; each
also returns the magnitudes that its rounding errors scale with."""

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


def norm_rope(x, weight, eps, cos, sin, rot, interleaved):
    """x [t][h][d], cos and sin [t][rot / 2]: (y, magnitude |a| + |b| per value)."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
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
