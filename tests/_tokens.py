"""Helpers of the token operators' tests: typed device arrays with chosen strides and alignment, their values in 64
bits, and the calls."""

import numpy as np
import torch

import conv2d_implicit_gemm_gb300 as ox
from tests._gpu import stream

KINDS = {"fp16": (torch.float16, ox.PRECISION_FP16), "bf16": (torch.bfloat16, ox.PRECISION_BF16),
         "fp32": (torch.float32, ox.PRECISION_FP32)}
# half a unit in the last place, relative; and the spacing of the smallest values
UNIT = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
TINY = {"fp16": 2.0 ** -25, "bf16": 0.0, "fp32": 0.0}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def strided(shape, kind, seed, pads=None, shift=0, scale=1.0, mean=0.0, fill=float("nan")):
    """Normal values in a view whose dimension i is pads[i] longer in memory, `shift` elements into its buffer; the
    memory around the view holds `fill`."""
    rng = np.random.default_rng(seed)
    pads = pads or [0] * len(shape)
    full = [n + p for n, p in zip(shape, pads)]
    buf = torch.full((int(np.prod(full)) + shift,), fill, dtype=KINDS[kind][0], device="cuda")
    view = buf[shift:].view(full)[tuple(slice(0, n) for n in shape)]
    view.copy_(torch.from_numpy(rng.standard_normal(shape) * scale + mean))
    return view


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def ptr(t):
    return 0 if t is None else t.data_ptr()


def linear(x, w, bias, residual, y, act, kind):
    m, k = x.shape
    n = w.shape[0]
    ox.oidnx_linear(ptr(x), x.stride(0), ptr(w), w.stride(0), ptr(bias), ptr(residual),
                    0 if residual is None else residual.stride(0), ptr(y), y.stride(0), m, n, k, ACTS.index(act),
                    KINDS[kind][1], stream())


def norm_rope(q, qo, k, ko, v, vo, qw, kw, eps, cos, sin, positions, slots, rot, interleaved, kind):
    def view(t):
        return (0, 0, 0) if t is None else (ptr(t), t.stride(0), t.stride(1))
    t, hq, d = q.shape
    ox.oidnx_qk_norm_rope(*view(q), *view(qo), *view(k), *view(ko), *view(v), *view(vo), ptr(qw), ptr(kw), eps, ptr(cos),
                          ptr(sin), 0 if cos is None else cos.shape[0], ptr(positions), ptr(slots), ko.shape[0], t, hq,
                          k.shape[1], d, rot, int(interleaved), KINDS[kind][1], stream())


def attention(q, k, v, o, lse, q_lens, kv_lens, window, sinks, scale, kind):
    b, tq, hq, d = q.shape
    cap, hk = k.shape[1:3]
    ox.oidnx_window_attention(ptr(q), *q.stride()[:3], ptr(k), *k.stride()[:3], ptr(v), *v.stride()[:3], ptr(o),
                              *o.stride()[:3], ptr(lse), ptr(q_lens), ptr(kv_lens), b, tq, cap, hq, hk, d, window,
                              sinks, scale, KINDS[kind][1], stream())


NORMS = ("none", "rms", "layer")
GATES = ("plain", "tanh", "sigmoid")


def block_norm(x, residual, total, y, post, post_weight, post_bias, pre, pre_weight, pre_bias, eps, gate, gate_act, scale,
               shift, groups, per, count, residual_scale, branch_scale, kind, total_kind):
    def row(t):
        return (0, 0) if t is None else (ptr(t), t.stride(0))
    t, n = x.shape
    ox.oidnx_block_norm(*row(x), *row(residual), *row(total), *row(y), NORMS.index(post), ptr(post_weight), ptr(post_bias),
                        NORMS.index(pre), ptr(pre_weight), ptr(pre_bias), eps, *row(gate), GATES.index(gate_act), *row(scale),
                        *row(shift), ptr(groups), per, count, residual_scale, branch_scale, t, n, KINDS[kind][1],
                        KINDS[total_kind][1], stream())


def norm_rope_axes(q, qo, k, ko, v, vo, norm, qw, kw, eps, cos, sin, positions, pair_axes, slots, interleaved, kind):
    def view(t):
        return (0, 0, 0) if t is None else (ptr(t), t.stride(0), t.stride(1))
    t, hq, d = q.shape
    ox.oidnx_qk_norm_rope_axes(*view(q), *view(qo), *view(k), *view(ko), *view(v), *view(vo), int(norm), ptr(qw), ptr(kw),
                               eps, ptr(cos), ptr(sin), 0 if cos is None else cos.shape[0], ptr(positions),
                               positions.stride(0), positions.shape[0], bytes(pair_axes), ptr(slots), ko.shape[0], t, hq,
                               k.shape[1], d, 2 * len(pair_axes), int(interleaved), KINDS[kind][1], stream())


def cross_attention(q, k, v, o, lse, q_lens, kv_lens, mask, scale, kind):
    b, tq, hq, d = q.shape
    kv, hk = k.shape[1:3]
    ox.oidnx_cross_attention(ptr(q), *q.stride()[:3], ptr(k), *k.stride()[:3], ptr(v), *v.stride()[:3], ptr(o),
                             *o.stride()[:3], ptr(lse), ptr(q_lens), ptr(kv_lens), ptr(mask),
                             0 if mask is None else mask.stride(0), b, tq, kv, hq, hk, d, scale, KINDS[kind][1], stream())


def done():
    ox.oidnx_token_sync_status(stream())
