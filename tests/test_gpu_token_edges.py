"""Edges of the token operators: activations at infinity, aligned rows that end within 16 bytes, prompts longer than a ring
holds, weights far below the largest, calls captured before they were ever made, memory kept, calls through ctypes
(tolerances and helpers of test_gpu_tokens.py)."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from oracle import tokens
from tests._tokens import ACTS, KINDS, TINY, UNIT, attention, done, f64, linear, norm_rope, strided
from tests.test_gpu_tokens import assert_within, check_attention, check_linear


# ---------------------------------------------------------------- infinities
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,k", [(4, 64), (4, 65), (33, 64), (33, 65), (180, 64), (180, 65)])
def test_linear_activations_at_infinity(m, k, act, kind):
    """Sums and biases of either infinity: what the definition gives (infinity, NaN or a number) at every value."""
    x, w, b = strided((m, k), kind, 1), strided((40, k), kind, 2), strided((40,), kind, 3)
    w[:, 5] = torch.where(torch.arange(40, device="cuda") % 2 == 0, 1.0, -1.0).to(w.dtype)
    x[1, 5], x[2, 5] = float("inf"), float("-inf")
    b[3], b[4], b[5] = float("inf"), float("-inf"), float("nan")
    y = torch.empty(m, 40, dtype=x.dtype, device="cuda")
    linear(x, w, b, None, y, act, kind)
    done()
    with np.errstate(invalid="ignore", over="ignore"):
        ref, _ = tokens.linear(f64(x), f64(w), f64(b), None, act)
    got = f64(y)
    for what in (np.isnan, np.isposinf, np.isneginf):
        np.testing.assert_array_equal(what(got), what(ref))


# ---------------------------------------------------------------- aligned rows that end within 16 bytes
@pytest.mark.parametrize("residual,inplace", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("n,pad", [(1, 7), (7, 1), (45, 3), (130, 6), (133, 131), (1001, 7)])
@pytest.mark.parametrize("m", [3, 40, 140, 600])
def test_linear_writes_no_value_behind_its_rows(m, n, pad, residual, inplace):
    """Rows of whole 16 bytes in memory, of which the output takes a part: what lies behind it stays."""
    check_linear(m, n, 64, "fp16" if m % 40 else "bf16", "gelu", residual=residual, inplace=inplace, pad=pad, seed=n)


@pytest.mark.parametrize("k,pad", [(1, 7), (7, 1), (45, 3), (130, 6), (133, 131)])
@pytest.mark.parametrize("m", [3, 40, 140, 600])
def test_linear_reads_no_value_behind_its_rows(m, k, pad):
    """The same of the operands: NaN lies behind each row."""
    check_linear(m, 72, k, "fp16", "none", pad=pad, seed=k)


# ---------------------------------------------------------------- prompts longer than the ring
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("b,tq,cap,kv,hq,hk,window,sinks", [
    (3, 512, 300, 512, 2, 2, 0, 0), (3, 1024, 600, 1024, 2, 2, 0, 0), (3, 1024, 600, 1024, 2, 2, 50, 0),
    (2, 700, 333, 5000, 4, 2, 40, 0), (3, 640, 200, 640, 2, 2, 0, 3), (3, 900, 150, 1000003, 6, 2, 20, 0)])
def test_attention_prompts_longer_than_the_ring(b, tq, cap, kv, hq, hk, window, sinks, d, kind):
    """Without sinks the first queries see nothing any more: o = 0, lse = -inf, also where they share a block with rows
    that do see keys."""
    check_attention(b, tq, cap, hq, hk, d, window, sinks, kind, kv_lens=[kv] * b, seed=cap + d)


@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("tq,cap", [(512, 300), (1024, 600), (4096, 2100)])
def test_attention_rows_before_the_ring_stay_zero(tq, cap, d):
    """The same call again and again: no row without a key ever holds anything but zeros."""
    q, k, v = strided((2, tq, 4, d), "bf16", 1), strided((2, cap, 4, d), "bf16", 2), strided((2, cap, 4, d), "bf16", 3)
    lens = torch.full((2,), tq, dtype=torch.int32, device="cuda")
    first = None
    for _ in range(30):
        o = torch.full_like(q, float("nan"))
        lse = torch.full((2, 4, tq), float("nan"), device="cuda")
        attention(q, k, v, o, lse, None, lens, 0, 0, d ** -0.5, "bf16")
        assert not o[:, :tq - cap].any() and torch.isneginf(lse[:, :, :tq - cap]).all()
        first = first or (o, lse)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    done()
    assert np.isfinite(first[1][:, :, tq - cap:].cpu().numpy()).all()


# ---------------------------------------------------------------- weights far below the largest
def check_one_loud_key(tq, b, n, d, gap, kind):
    """The first key's score is `gap` above all the others' and its value zero, so that the output is the others' alone.

    Tolerance, relative to the output (all weights but one are equal): the result's rounding and that of the weights,
    UNIT each, twice the latter for the mean; scores of at most gap, in base 2, off by 2^-22 of them; exponentials 2^-20.
    fp16 weights are held against 2^7 or more times the largest (2^-24 is the spacing of the smallest there): 2^-32 each
    against e^-gap."""
    q = torch.ones(b, tq, 2, d, dtype=KINDS[kind][0], device="cuda")
    k = torch.zeros(b, n, 1, d, dtype=KINDS[kind][0], device="cuda")
    k[:, 0, :, 0] = gap
    v = strided((b, n, 1, d), kind, 1, mean=512.0, scale=64.0)
    v[:, 0] = 0
    o, lse = torch.empty_like(q), torch.empty(b, 2, tq, device="cuda")
    attention(q, k, v, o, lse, None, None, 0, 0, 1.0, kind)
    done()
    ref, ref_lse, mag, dots = tokens.window_attention(f64(q), f64(k), f64(v), [tq] * b, [n] * b, 0, 0, 1.0)
    small = 2.0 ** -32 * np.exp(gap) if kind == "fp16" else 0.0
    tol = (3 * UNIT[kind] + 2.0 ** -22 * gap * 2 + 2.0 ** -20 + small) * np.abs(ref) + TINY[kind]
    assert_within(f64(o), ref, tol)
    assert_within(lse.double().cpu().numpy(), ref_lse, np.full(ref_lse.shape, 2.0 ** -18))


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("gap", [10.0, 14.0, 16.875, 18.0])
@pytest.mark.parametrize("d", [64, 80, 128])
def test_attention_of_prompts_far_below_the_largest_score(d, gap, kind):
    check_one_loud_key(500, 6, 1500, d, gap, kind)


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("gap", [10.0, 14.0, 16.875, 18.0])
@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("b,tq,n", [(2, 1, 16), (2, 1, 2000), (200, 1, 17), (3, 20, 60)])
def test_attention_of_few_queries_far_below_the_largest_score(b, tq, n, d, gap, kind):
    check_one_loud_key(tq, b, n, d, gap, kind)


# ---------------------------------------------------------------- graph capture
CAPTURE = """
import sys
sys.path.insert(0, {root!r})
import torch
from tests._tokens import attention, done, linear, norm_rope, strided

def product(m, n, k, shift=0):
    x, w = strided((m, k), "bf16", 1, None, shift), strided((n, k), "bf16", 2, None, shift)
    y = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    return y, lambda: linear(x, w, None, None, y, "silu", "bf16")

def window(tq, cap, hq, hk, d):
    q, k = strided((1, tq, hq, d), "bf16", 3), strided((1, cap, hk, d), "bf16", 4)
    o = torch.zeros_like(q)
    return o, lambda: attention(q, k, k, o, None, None, None, 300, 4, 0.125, "bf16")

def norm(d):
    q, k = strided((3, 4, d), "bf16", 5), strided((3, 2, d), "bf16", 6)
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    return qo, lambda: norm_rope(q, qo, k, ko, None, None, None, None, 1e-6, None, None, None, None, 0, False, "bf16")

calls = [product(9, 256, 256), product(60, 256, 512), product(128, 256, 2048), product(9, 256, 255),
         product(100, 64, 255, 1), product(200, 64, 255, 1), product(300, 200, 256), product(3000, 3000, 512),
         window(1, 900, 8, 2, 64), window(1, 900, 8, 2, 128), window(20, 90, 2, 2, 128), window(600, 900, 8, 2, 64),
         window(600, 900, 8, 2, 128), window(3, 90, 2, 1, 63), window(3, 90, 2, 1, 256), norm(64), norm(72), norm(65)]
norm(128)[1]()  # the one call on the device
done()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for out, call in calls:
        call()
for _ in range(2):
    graph.replay()
    torch.cuda.synchronize()
    got = [out.clone() for out, call in calls]
    for out, call in calls:
        out.zero_()
for (out, call), g in zip(calls, got):
    call()
    done()
    assert g.any() and torch.equal(g, out)
print("captured")
"""


def test_every_form_can_be_captured_once_any_call_has_been_made():
    """In a process of its own, whose one call before the capture is a norm."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", CAPTURE.format(root=root)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "captured" in run.stdout, run.stderr[-2000:]


# ---------------------------------------------------------------- memory
def test_memory_of_a_large_unaligned_product_is_given_back():
    """Copies of 3 GiB: of these at most 1 GiB stays with the library once the GPU has been waited for."""
    m, k = 3 * 2 ** 20, 511
    x, w = torch.zeros(m, k, dtype=torch.float16, device="cuda"), torch.zeros(8, k, dtype=torch.float16, device="cuda")
    y = torch.empty(m, 8, dtype=torch.float16, device="cuda")
    linear(x[:64], w, None, None, y[:64], "none", "fp16")
    done()
    before = torch.cuda.mem_get_info()[0]
    linear(x, w, None, None, y, "none", "fp16")
    done()
    assert before - torch.cuda.mem_get_info()[0] <= 1 << 30
    assert not y.any()


# ---------------------------------------------------------------- entries
def test_calls_through_ctypes_give_the_same_results(monkeypatch):
    """What the package does without its extension module."""
    import conv2d_implicit_gemm_gb300 as ox
    from conv2d_implicit_gemm_gb300 import _calls_ctypes
    x, w = strided((9, 256), "bf16", 1), strided((64, 256), "bf16", 2)
    q, k = strided((3, 5, 8, 64), "bf16", 3), strided((3, 70, 2, 64), "bf16", 4)
    results = []
    for calls in (ox._calls, _calls_ctypes.bind(ox._lib)):
        monkeypatch.setattr(ox, "_calls", calls)
        y, o, lse = torch.empty(9, 64, dtype=x.dtype, device="cuda"), torch.empty_like(q), torch.empty(3, 8, 5, device="cuda")
        qo, ko = torch.empty_like(q[0]), torch.empty_like(k[0])
        linear(x, w, None, None, y, "silu", "bf16")
        attention(q, k, k, o, lse, None, None, 30, 2, 0.125, "bf16")
        norm_rope(q[0], qo, k[0, :5], ko, None, None, None, None, 1e-6, None, None, None, None, 0, False, "bf16")
        done()
        results.append((y, o, lse, qo, ko[:5]))
    assert all(torch.equal(a, b) for a, b in zip(*results))
