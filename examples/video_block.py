"""A conditioned block over the tokens of a video clip, from the library's calls.

The tokens of `frames` maps of rows x cols attend to one another (heads turned by time, height and width), then to the
states of an encoder (a text of its own length for each clip, with a mask), and go through a feed-forward pair.  Each
branch ends in one call that norms it, gates it, adds it to the sum of all branches so far (held in fp32) and norms that
for the next branch, with the scales and shifts that a condition (the time step, say) gives each clip.

    python examples/video_block.py            # random weights; checks against the same block in plain torch in 64 bits
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import conv2d_implicit_gemm_gb300 as ox

PRECISION = {torch.float16: ox.PRECISION_FP16, torch.bfloat16: ox.PRECISION_BF16}
EPS = 1e-6


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _stream():
    return torch.cuda.current_stream().cuda_stream


def linear(x, w, bias=None, act=ox.ACT_NONE):
    m, (n, k) = x.numel() // x.shape[-1], w.shape
    y = torch.empty(*x.shape[:-1], n, dtype=x.dtype, device=x.device)
    ox.oidnx_linear(x.data_ptr(), k, w.data_ptr(), k, _ptr(bias), 0, n, y.data_ptr(), n, m, n, k, act, PRECISION[x.dtype],
                    _stream())
    return y


def attend(q, k, v, mask=None):
    """q [b][t][hq][d] to k and v [b][n][hk][d]; mask [b][n] of bytes."""
    (b, t, hq, d), (n, hk) = q.shape, k.shape[1:3]
    o = torch.empty(b, t, hq, d, dtype=q.dtype, device=q.device)
    ox.oidnx_cross_attention(q.data_ptr(), *q.stride()[:3], k.data_ptr(), *k.stride()[:3], v.data_ptr(), *v.stride()[:3],
                             o.data_ptr(), *o.stride()[:3], 0, 0, 0, _ptr(mask), n, b, t, n, hq, hk, d, d ** -0.5,
                             PRECISION[q.dtype], _stream())
    return o.view(b, t, hq * d)


class VideoBlock:
    """Random weights of one block."""

    def __init__(self, channels=512, heads=8, key_heads=8, head=64, text=256, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weight(n, k):
            return (torch.randn(n, k, generator=g, device="cuda") / k ** 0.5).to(dtype)

        def ones(n):
            return (1 + 0.1 * torch.randn(n, generator=g, device="cuda")).to(dtype)

        self.heads, self.key_heads, self.head, self.dtype = heads, key_heads, head, dtype
        self.qkv, self.out = weight((heads + 2 * key_heads) * head, channels), weight(channels, heads * head)
        self.q_weight, self.k_weight = ones(head), ones(head)
        self.cross_q, self.cross_out = weight(heads * head, channels), weight(channels, heads * head)
        self.cross_k, self.cross_v = weight(key_heads * head, text), weight(key_heads * head, text)
        self.up, self.down = weight(4 * channels, channels), weight(channels, 4 * channels)
        self.before = [ones(channels) for _ in range(4)]  # of the self attention, the text, the feed-forward pair, what follows
        self.after = [ones(channels) for _ in range(3)]
        pairs = head // 2
        self.sections = [pairs - 2 * (3 * pairs // 8), 3 * pairs // 8, 3 * pairs // 8]  # of time, height and width
        self.pair_axes = bytes(a for a, n in enumerate(self.sections) for _ in range(n))
        angle = torch.arange(256, device="cuda", dtype=torch.float64)[:, None] * (
            10000.0 ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs))
        self.cos, self.sin = angle.cos().float().contiguous(), angle.sin().float().contiguous()

    def step(self, branch, total, before, after, gate, scale, shift):
        """(total + gate norm(branch), its norm with scale and shift); the first step has no total yet and no norm."""
        b, t, c = branch.shape
        new = torch.empty(b, t, c, dtype=torch.float32, device="cuda") if total is None else total
        y = torch.empty_like(branch)
        ox.oidnx_block_norm(branch.data_ptr(), c, _ptr(total), c, new.data_ptr(), c, y.data_ptr(), c,
                            ox.NORM_NONE if after is None else ox.NORM_RMS, _ptr(after), 0, ox.NORM_RMS, before.data_ptr(), 0,
                            EPS, _ptr(gate), c, ox.GATE_TANH, _ptr(scale), c, _ptr(shift), c, 0, t, b, 1.0, 1.0, b * t, c,
                            PRECISION[self.dtype], ox.PRECISION_FP32, _stream())
        return new, y

    def __call__(self, x, shape, condition, text, mask):
        """x [b][frames x rows x cols][channels]; condition [7][b][channels]: scale and shift before the self attention and
        the feed-forward pair, the gates of the three branches; text [b][n][..]; mask [b][n] of bytes."""
        b, t, _ = x.shape
        frames, rows, cols = shape
        hq, hk, d, row = self.heads, self.key_heads, self.head, (self.heads + 2 * self.key_heads) * self.head
        i = torch.arange(t, device="cuda")
        positions = torch.stack((i // (rows * cols), i // cols % rows, i % cols)).to(torch.int32).repeat(1, b)
        total, y = self.step(x, None, self.before[0], None, None, condition[0], condition[1])

        qkv = linear(y, self.qkv)
        q, k, v = (torch.empty(b, t, h, d, dtype=x.dtype, device="cuda") for h in (hq, hk, hk))
        base, size = qkv.data_ptr(), qkv.element_size()
        ox.oidnx_qk_norm_rope_axes(base, row, d, q.data_ptr(), hq * d, d, base + hq * d * size, row, d, k.data_ptr(), hk * d, d,
                                   base + (hq + hk) * d * size, row, d, v.data_ptr(), hk * d, d, 1, self.q_weight.data_ptr(),
                                   self.k_weight.data_ptr(), EPS, self.cos.data_ptr(), self.sin.data_ptr(), self.cos.shape[0],
                                   positions.data_ptr(), b * t, 3, self.pair_axes, 0, b * t, b * t, hq, hk, d, d, 0,
                                   PRECISION[x.dtype], _stream())
        total, y = self.step(linear(attend(q, k, v), self.out), total, self.before[1], self.after[0], condition[4], None, None)

        n = text.shape[1]
        keys, values = (linear(text, w).view(b, n, hk, d) for w in (self.cross_k, self.cross_v))
        a = attend(linear(y, self.cross_q).view(b, t, hq, d), keys, values, mask)
        total, y = self.step(linear(a, self.cross_out), total, self.before[2], self.after[1], condition[5], condition[2],
                             condition[3])
        a = linear(linear(y, self.up, None, ox.ACT_GELU_TANH), self.down)
        return self.step(a, total, self.before[3], self.after[2], condition[6], None, None)

    def plain(self, x, shape, condition, text, mask):
        """The same in plain torch, in 64 bits."""
        b, t, _ = x.shape
        frames, rows, cols = shape
        hq, hk, d = self.heads, self.key_heads, self.head
        x, text = x.double(), text.double()
        cond = [z.double()[:, None] for z in condition]

        def norm(z, w):
            return z * (z.pow(2).mean(-1, keepdim=True) + EPS).rsqrt() * w.double()

        def attention(q, k, v, seen):
            k, v = (z.repeat_interleave(hq // hk, 2) for z in (k, v))
            score = torch.einsum("bihd,bjhd->bhij", q, k) * d ** -0.5
            if seen is not None:
                score = score.masked_fill(seen[:, None, None] == 0, float("-inf"))
            weight = score.softmax(-1)
            if seen is not None:  # a text of no words adds nothing
                weight = torch.where((seen != 0).any(-1)[:, None, None, None], weight, 0.0)
            return torch.einsum("bhij,bjhd->bihd", weight, v).reshape(b, t, hq * d)

        i = torch.arange(t, device="cuda")
        places = torch.stack((i // (rows * cols), i // cols % rows, i % cols))
        axis = torch.tensor(list(self.pair_axes), device="cuda")
        at, pair = places[axis].t(), torch.arange(d // 2, device="cuda")
        turn = torch.complex(self.cos[at, pair].double(), self.sin[at, pair].double())[None, :, None]

        def turned(z, w):
            z = norm(z, w)
            z = torch.complex(z[..., :d // 2], z[..., d // 2:]) * turn
            return torch.cat((z.real, z.imag), -1)

        y = norm(x, self.before[0]) * (1 + cond[0]) + cond[1]
        qkv = (y @ self.qkv.double().t()).view(b, t, hq + 2 * hk, d)
        a = attention(turned(qkv[:, :, :hq], self.q_weight), turned(qkv[:, :, hq:hq + hk], self.k_weight), qkv[:, :, hq + hk:], None)
        x = x + cond[4].tanh() * norm(a @ self.out.double().t(), self.after[0])
        y = norm(x, self.before[1])
        n = text.shape[1]
        keys, values = ((text @ w.double().t()).view(b, n, hk, d) for w in (self.cross_k, self.cross_v))
        a = attention((y @ self.cross_q.double().t()).view(b, t, hq, d), keys, values, mask)
        x = x + cond[5].tanh() * norm(a @ self.cross_out.double().t(), self.after[1])
        y = norm(x, self.before[2]) * (1 + cond[2]) + cond[3]
        a = torch.nn.functional.gelu(y @ self.up.double().t(), approximate="tanh") @ self.down.double().t()
        x = x + cond[6].tanh() * norm(a, self.after[2])
        return x, norm(x, self.before[3])


def inputs(block, batch, shape, length, seed=1):
    """Random tokens, condition, texts and a mask that ends each text elsewhere."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t, c = shape[0] * shape[1] * shape[2], block.qkv.shape[1]

    def normal(*size, scale=1.0):
        return (torch.randn(*size, generator=g, device="cuda") * scale).to(block.dtype)

    mask = (torch.arange(length, device="cuda")[None] < torch.arange(1, batch + 1, device="cuda")[:, None] * length // batch)
    return (normal(batch, t, c), shape, normal(7, batch, c, scale=0.5), normal(batch, length, block.cross_k.shape[1]),
            mask.to(torch.uint8).contiguous())


def run(batch=2, shape=(3, 12, 20), length=77, dtype=torch.bfloat16, **sizes):
    """Relative differences of the sum and of its norm from the 64-bit block, of the worst token."""
    block = VideoBlock(dtype=dtype, **sizes)
    given = inputs(block, batch, shape, length)
    got, ref = block(*given), block.plain(*given)
    ox.oidnx_token_sync_status(_stream())
    return [((a.double() - b).norm(dim=-1) / b.norm(dim=-1)).max().item() for a, b in zip(got, ref)]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--frames", type=int, default=8)
    ap.add_argument("--rows", type=int, default=34)
    ap.add_argument("--cols", type=int, default=60)
    ap.add_argument("--text", type=int, default=77)
    a = ap.parse_args()
    total, normed = run()
    print(f"against 64 bits, worst token: sum {total:.2e}, its norm {normed:.2e}")
    block = VideoBlock(channels=1024, heads=16, key_heads=16)
    given = inputs(block, 1, (a.frames, a.rows, a.cols), a.text)
    for _ in range(3):
        block(*given)
    torch.cuda.synchronize()
    begin = time.perf_counter()
    for _ in range(10):
        block(*given)
    torch.cuda.synchronize()
    print(f"{a.frames} maps of {a.rows} x {a.cols} tokens, 1024 channels: {(time.perf_counter() - begin) * 1e2:.3f} ms")


if __name__ == "__main__":
    main()
