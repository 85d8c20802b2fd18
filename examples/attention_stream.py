"""An attention block over endless token streams, from the token operators.

Each stream sends a few tokens at a time (a few for each frame, say); random ones here.  A step projects
them to queries, keys and values (oidnx_linear), norms and rotates the heads and appends keys and values to the stream's
ring cache (oidnx_qk_norm_rope), attends over the first tokens and a sliding window (oidnx_window_attention), and ends in
the output projection and a feed-forward pair, each with its residual in the same call.  The cache holds
sinks + window + step - 1 slots however long the stream runs.

    python examples/attention_stream.py            # a prompt, then single tokens; checks against one pass over everything
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import conv2d_implicit_gemm_gb300 as ox

PRECISION = {torch.float16: ox.PRECISION_FP16, torch.bfloat16: ox.PRECISION_BF16}


def linear(x, w, bias=None, act=ox.ACT_NONE, residual=None):
    """act(x w^T + bias) + residual over the last dimension."""
    m, (n, k) = x.numel() // x.shape[-1], w.shape
    y = torch.empty(*x.shape[:-1], n, dtype=x.dtype, device=x.device)
    ox.oidnx_linear(x.data_ptr(), k, w.data_ptr(), k, 0 if bias is None else bias.data_ptr(),
                    0 if residual is None else residual.data_ptr(), n, y.data_ptr(), n, m, n, k, act, PRECISION[x.dtype],
                    torch.cuda.current_stream().cuda_stream)
    return y


class AttentionBlock:
    """Random weights of one block, and the ring caches of `streams` streams."""

    def __init__(self, channels=512, heads=8, key_heads=2, head=64, window=256, sinks=4, step=64, streams=2, longest=8192,
                 capacity=None, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weight(n, k):
            return (torch.randn(n, k, generator=g, device="cuda") / k ** 0.5).to(dtype)

        self.heads, self.key_heads, self.head, self.window, self.sinks = heads, key_heads, head, window, sinks
        self.streams, self.capacity = streams, capacity or sinks + window + step - 1
        self.step_tokens = step
        self.qkv = weight((heads + 2 * key_heads) * head, channels)
        self.out = weight(channels, heads * head)
        self.up, self.down = weight(4 * channels, channels), weight(channels, 4 * channels)
        self.up_bias = (torch.randn(4 * channels, generator=g, device="cuda") * 0.1).to(dtype)
        self.q_weight = (1 + 0.1 * torch.randn(head, generator=g, device="cuda")).to(dtype)
        self.k_weight = (1 + 0.1 * torch.randn(head, generator=g, device="cuda")).to(dtype)
        angle = torch.arange(longest, device="cuda", dtype=torch.float64)[:, None] * (
            10000.0 ** (-torch.arange(0, head, 2, device="cuda", dtype=torch.float64) / head))
        self.cos, self.sin = angle.cos().float().contiguous(), angle.sin().float().contiguous()
        shape = (streams, self.capacity, key_heads, head)
        self.k_cache = torch.empty(shape, dtype=dtype, device="cuda")
        self.v_cache = torch.empty(shape, dtype=dtype, device="cuda")
        self.written = 0  # tokens of each stream so far

    def __call__(self, x):
        """x: [streams][tokens][channels], the next tokens of every stream."""
        b, t, _ = x.shape
        assert b == self.streams and t <= self.step_tokens, "more tokens than the ring has room for"
        hq, hk, d, row = self.heads, self.key_heads, self.head, (self.heads + 2 * self.key_heads) * self.head
        stream = torch.cuda.current_stream().cuda_stream
        precision = PRECISION[x.dtype]

        at = torch.arange(self.written, self.written + t, device="cuda", dtype=torch.int32)
        ring = self.capacity - self.sinks
        slot = torch.where(at < self.capacity, at, self.sinks + (at - self.sinks) % ring)
        slots = (slot + torch.arange(b, device="cuda", dtype=torch.int32)[:, None] * self.capacity).to(torch.int32)
        positions = at.repeat(b)
        self.written += t
        lens = torch.full((b,), self.written, device="cuda", dtype=torch.int32)

        qkv = linear(x, self.qkv)
        q = torch.empty(b, t, hq, d, dtype=x.dtype, device="cuda")
        base, size = qkv.data_ptr(), qkv.element_size()
        ox.oidnx_qk_norm_rope(base, row, d, q.data_ptr(), hq * d, d,
                              base + hq * d * size, row, d, self.k_cache.data_ptr(), hk * d, d,
                              base + (hq + hk) * d * size, row, d, self.v_cache.data_ptr(), hk * d, d,
                              self.q_weight.data_ptr(), self.k_weight.data_ptr(), 1e-6, self.cos.data_ptr(),
                              self.sin.data_ptr(), self.cos.shape[0], positions.data_ptr(), slots.data_ptr(),
                              b * self.capacity, b * t, hq, hk, d, d, 0, precision, stream)
        o = torch.empty_like(q)
        ox.oidnx_window_attention(q.data_ptr(), *q.stride()[:3], self.k_cache.data_ptr(), *self.k_cache.stride()[:3],
                                  self.v_cache.data_ptr(), *self.v_cache.stride()[:3], o.data_ptr(), *o.stride()[:3], 0, 0,
                                  lens.data_ptr(), b, t, self.capacity, hq, hk, d, self.window, self.sinks, d ** -0.5,
                                  precision, stream)
        x = linear(o.view(b, t, hq * d), self.out, residual=x)
        return linear(linear(x, self.up, self.up_bias, ox.ACT_GELU_TANH), self.down, residual=x)


def run(tokens=600, prompt_step=64, singles=20, streams=2, dtype=torch.bfloat16, **sizes):
    """Streams in steps and then single tokens over a ring, against one call over a cache that holds everything; returns
    the largest relative difference of a token's output."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    ring = AttentionBlock(step=prompt_step, streams=streams, dtype=dtype, **sizes)
    whole = AttentionBlock(step=tokens, streams=streams, dtype=dtype, capacity=tokens, **sizes)
    x = torch.randn(streams, tokens, ring.qkv.shape[1], generator=g, device="cuda").to(dtype)
    parts, at = [], 0
    while at < tokens:
        step = 1 if at >= tokens - singles else min(prompt_step, tokens - singles - at)
        parts.append(ring(x[:, at:at + step].contiguous()))
        at += step
    ref = whole(x)
    ox.oidnx_token_sync_status(torch.cuda.current_stream().cuda_stream)
    got = torch.cat(parts, 1)
    return ((got.double() - ref.double()).norm(dim=-1) / ref.double().norm(dim=-1)).max().item()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=2000)
    ap.add_argument("--streams", type=int, default=4)
    ap.add_argument("--window", type=int, default=512)
    a = ap.parse_args()
    off = run(tokens=a.tokens, streams=a.streams, window=a.window)
    print(f"{a.streams} streams of {a.tokens} tokens, window {a.window}: in steps and at once differ by {off:.2e} (relative, "
          "worst token)")
    block = AttentionBlock(step=64, streams=a.streams, window=a.window)
    x = torch.randn(a.streams, 1, 512, device="cuda").to(torch.bfloat16)
    for _ in range(5):
        block(x)
    torch.cuda.synchronize()
    begin = time.perf_counter()
    for _ in range(100):
        block(x)
    torch.cuda.synchronize()
    print(f"one token a stream: {(time.perf_counter() - begin) * 1e4:.1f} us a step")


if __name__ == "__main__":
    main()
