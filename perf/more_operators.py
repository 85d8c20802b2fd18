"""Workloads of a conditioned block over the tokens of images and video: the norms before and after a branch with its
gate and residual, the norm and rotation of heads by positions of several axes, and attention to an encoder's states.
Each case is one operator at one size; run() makes the pass with the library's calls (own) or in plain torch operations
in 32 bits."""

import math

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
NORMS = ("none", "rms", "layer")
GATES = ("plain", "tanh", "sigmoid")
EPS = 1e-6


def listed():
    return [
        # one token of a stream between two blocks: norm after, gate and residual, norm before; the smallest call
        dict(name="block_token", op="block", t=1, n=4096, post="rms", pre="rms", gate="channel", gate_act="plain",
             modulate=False, residual=True, bias=False, alpha=1.0, beta=1.0, per=1, type="bf16", stream="bf16"),
        # the tokens of a frame's bottleneck map (1920x1080 / 32: 60 x 34), an odd channel count, the modulation of two images
        dict(name="block_odd", op="block", t=4080, n=1001, post="none", pre="layer", gate="groups", gate_act="plain",
             modulate=True, residual=True, bias=True, alpha=1.0, beta=1.0, per=2040, type="fp16", stream="fp16"),
        # sixteen frames of that map through a sandwich of norms, the sum of all branches held in fp32
        dict(name="block_video", op="block", t=32640, n=1536, post="rms", pre="rms", gate="groups", gate_act="tanh",
             modulate=True, residual=True, bias=False, alpha=1.0, beta=1.0, per=2040, type="bf16", stream="fp32"),
        # a long prompt, everything in 16 bits, the branch scaled
        dict(name="block_prompt", op="block", t=16384, n=4096, post="rms", pre="rms", gate="channel", gate_act="plain",
             modulate=False, residual=True, bias=False, alpha=1.0, beta=0.22, per=16384, type="bf16", stream="bf16"),
        # one new token of one stream, its positions in time, height and width
        dict(name="axes_token", op="axes", frames=1, rows=1, cols=1, hq=32, hk=8, d=128, sections="16 24 24",
             mixed=False, interleaved=False, norm=True, weight=True, cache=512, type="bf16"),
        # one map, two axes of adjacent pairs, heads that no power of two divides, no norm
        dict(name="axes_map", op="axes", frames=1, rows=34, cols=60, hq=7, hk=7, d=72, sections="18 18", mixed=False,
             interleaved=True, norm=False, weight=False, cache=0, type="fp16"),
        # sixteen frames, the axes taking turns over the pairs, keys and values appended to the cache
        dict(name="axes_video", op="axes", frames=16, rows=34, cols=60, hq=16, hk=16, d=128, sections="22 21 21",
             mixed=True, interleaved=False, norm=True, weight=True, cache=32768, type="bf16"),
        # one token of one stream that reads a long encoding
        dict(name="cross_token", op="cross", b=1, tq=1, kv=20000, hq=32, hk=8, d=128, ragged=False, mask=False,
             type="bf16"),
        # one token each of many streams, encodings of all lengths
        dict(name="cross_tokens", op="cross", b=64, tq=1, kv=1500, hq=20, hk=20, d=64, ragged=True, mask=False,
             type="fp16"),
        # the tokens of four maps (1920x1080 / 16: 120 x 68) that read a short text
        dict(name="cross_text", op="cross", b=4, tq=8160, kv=77, hq=16, hk=16, d=64, ragged=False, mask=False,
             type="fp16"),
        # two texts one behind the other, each padded, shared heads that fill no tile
        dict(name="cross_mask", op="cross", b=5, tq=700, kv=333, hq=6, hk=2, d=80, ragged=True, mask=True, type="fp16"),
        # a video's tokens that read a whole map's
        dict(name="cross_long", op="cross", b=1, tq=8160, kv=8160, hq=16, hk=16, d=128, ragged=False, mask=False,
             type="bf16"),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("block", "axes", "cross"))
    kind = rng.choice(("fp16", "bf16"))
    if op == "block":
        kind = rng.choice(("fp16", "bf16", "fp32"))
        n = _log(rng, 64, 16384)
        if rng.random() < 0.7:  # the usual widths; the others stay odd
            n = (n + 7) // 8 * 8
        t = rng.choice((1, _log(rng, 1, 64), _log(rng, 64, 32768)))
        t = min(t, max(1, 30_000_000 // n))
        return dict(op=op, t=t, n=n, post=rng.choice(NORMS), pre=rng.choice(("rms", "layer")),
                    gate=rng.choice(("none", "channel", "groups")), gate_act=rng.choice(GATES),
                    modulate=rng.random() < 0.5, residual=rng.random() < 0.8, bias=rng.random() < 0.3,
                    alpha=rng.choice((1.0, 1.0, round(rng.uniform(0.5, 2.0), 3))),
                    beta=rng.choice((1.0, 1.0, round(rng.uniform(0.1, 1.0), 3))),
                    per=rng.choice((1, rng.randint(1, t), t)) if t * n < 4_000_000 else rng.randint((t + 15) // 16, t),
                    type=kind, stream=rng.choice((kind, "fp32")))
    if op == "axes":
        kind = rng.choice(("fp16", "bf16", "fp32"))
        d = rng.choice((64, 128, 128, 8 * rng.randint(4, 32)))
        hk = rng.randint(1, 8)
        hq = hk * rng.choice((1, 2, 4))
        rows, cols = rng.choice(((1, 1), (_log(rng, 1, 64), _log(rng, 1, 64))))
        frames = rng.choice((1, _log(rng, 1, 64)))
        most = 150_000_000 // (d * (hq + 2 * hk) * (4 if kind == "fp32" else 2))
        frames = max(1, min(frames, most // (rows * cols)))
        pairs = rng.choice((d, d // 4 * 2)) // 2
        axes = rng.randint(2, 4)
        cuts = sorted(rng.randint(0, pairs) for _ in range(axes - 1))
        sections = " ".join(str(b - a) for a, b in zip([0] + cuts, cuts + [pairs]))
        t = frames * rows * cols
        norm = rng.random() < 0.7
        return dict(op=op, frames=frames, rows=rows, cols=cols, hq=hq, hk=hk, d=d, sections=sections,
                    mixed=rng.random() < 0.4, interleaved=rng.random() < 0.5, norm=norm, weight=norm and rng.random() < 0.7,
                    cache=rng.choice((0, t + rng.randint(0, 512))), type=kind)
    d = rng.choice((64, 128, 128, 8 * rng.randint(4, 20)))
    hk = rng.randint(1, 16)
    if rng.random() < 0.5:  # tokens
        b, group = _log(rng, 1, 64), rng.choice((1, 1, 4, 8))
        kv = _log(rng, 16, min(32768, 300_000_000 // (b * hk * d * 4)))
        return dict(op=op, b=b, tq=rng.choice((1, 1, 1, rng.randint(2, 8))), kv=kv, hq=hk * group, hk=hk, d=d,
                    ragged=rng.random() < 0.5, mask=rng.random() < 0.3, type=kind)
    group = rng.choice((1, 1, 1, 4))
    b, tq = rng.randint(1, 4), _log(rng, 16, 8192)
    if b * tq * hk * group * d > 60_000_000:
        b, hk = 1, min(hk, 4)
    kv = _log(rng, 16, max(16, min(8192, 500_000_000 // (b * tq * hk * group))))
    return dict(op=op, b=b, tq=tq, kv=kv, hq=hk * group, hk=hk, d=d, ragged=rng.random() < 0.4,
                mask=rng.random() < 0.3, type=kind)


def _lengths(case):
    """(query length, key length) of each sequence; ragged batches hold short and empty ones among the full."""
    b, tq, kv = case["b"], case["tq"], case["kv"]
    if not case["ragged"]:
        return [(tq, kv)] * b
    return [(tq if i % 2 == 0 else max(1, tq * 5 // 7),
             kv if i == 0 else 0 if i == 3 else max(1, kv * ((i * 37 + 11) % 64) // 64)) for i in range(b)]


def _seen(case):
    """The keys that a sequence's queries see, as lists of positions: up to its length and, with a mask, the written
    parts of two texts of half of it each."""
    got = []
    for i, (_, n) in enumerate(_lengths(case)):
        half = n // 2
        first, second = half * ((i * 29 + 17) % 32) // 32, (n - half) * ((i * 23 + 31) % 32) // 32
        got.append(list(range(first)) + list(range(half, half + second)) if case["mask"] else list(range(n)))
    return got


def _sections(case):
    """Rotation pairs of each axis."""
    return [int(n) for n in case["sections"].split()]


def _pair_axes(case):
    """The axis of each rotation pair: sections one after the other, or (mixed) in turns while their pairs last."""
    sections = _sections(case)
    if not case["mixed"]:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    return [a for turn in range(max(sections)) for a, n in enumerate(sections) if turn < n]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind = TYPES[case["type"]]

    def normal(*shape, scale=1.0, mean=0.0, kind=kind):
        return (torch.randn(*shape, generator=g, device="cuda") * scale + mean).to(kind)

    s = {"case": dict(case)}
    if case["op"] == "block":
        t, n = case["t"], case["n"]
        groups = (t + case["per"] - 1) // case["per"]
        s["x"] = normal(t, n, scale=2.0, mean=0.1)
        s["residual"] = normal(t, n, scale=3.0, kind=TYPES[case["stream"]]) if case["residual"] else None
        for name, norm in (("post", case["post"]), ("pre", case["pre"])):
            s[name + "_weight"] = normal(n, scale=0.2, mean=1.0) if norm != "none" else None
            s[name + "_bias"] = normal(n, scale=0.1) if norm != "none" and case["bias"] else None
        s["gate"] = None
        if case["gate"] != "none":
            s["gate"] = normal(1 if case["gate"] == "channel" else groups, n, scale=0.3, mean=0.5)
        s["scale"] = normal(groups, n, scale=0.3) if case["modulate"] else None
        s["shift"] = normal(groups, n, scale=0.3) if case["modulate"] else None
    elif case["op"] == "axes":
        frames, rows, cols, hq, hk, d = (case[x] for x in ("frames", "rows", "cols", "hq", "hk", "d"))
        t, sections = frames * rows * cols, _sections(case)
        pairs = sum(sections)
        s["qkv"] = normal(t, hq + 2 * hk, d, scale=1.5)  # as one projection wrote them
        s["q_weight"] = normal(d, scale=0.2, mean=1.0) if case["weight"] else None
        s["k_weight"] = normal(d, scale=0.2, mean=1.0) if case["weight"] else None
        begin = int(torch.randint(0, 64, (1,), generator=g, device="cuda").item())
        i = torch.arange(t, device="cuda")
        places = [begin + i // (rows * cols), i // cols % rows, i % cols, i * 0 + begin]
        s["positions"] = torch.stack(places[:len(sections)]).to(torch.int32)
        s["pair_axes"] = bytes(_pair_axes(case))
        longest = max(frames, rows, cols) + 64
        angle = torch.arange(longest, device="cuda", dtype=torch.float64)[:, None] * (
            10000.0 ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs))
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        if case["cache"]:
            s["slots"] = ((i + begin) % case["cache"]).to(torch.int32)
            s["k_cache"], s["v_cache"] = normal(case["cache"], hk, d), normal(case["cache"], hk, d)
    else:
        b, tq, kv, hq, hk, d = (case[x] for x in ("b", "tq", "kv", "hq", "hk", "d"))
        s["q"] = normal(b, tq, hq, d, scale=1.2)
        s["k"], s["v"] = normal(b, kv, hk, d, scale=1.2), normal(b, kv, hk, d)
        lengths, seen = _lengths(case), torch.zeros(b, kv, dtype=torch.bool)
        for row, keys in zip(seen, _seen(case)):
            row[keys] = True
        for i, (_, n) in enumerate(lengths):  # places behind a sequence's last key hold anything
            s["k"][i, n:] = float("nan")
            s["v"][i, n:] = float("nan")
        s["mask"] = seen.to(torch.uint8).cuda() if case["mask"] else None
        s["q_lens"] = torch.tensor([q for q, _ in lengths], dtype=torch.int32, device="cuda") if case["ragged"] else None
        s["kv_lens"] = torch.tensor([n for _, n in lengths], dtype=torch.int32, device="cuda") if case["ragged"] else None
        s["factor"] = 1 / math.sqrt(d)
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return {"block": _block_own, "axes": _axes_own, "cross": _cross_own}[op](s)
    return {"block": _block_plain, "axes": _axes_plain, "cross": _cross_plain}[op](s)


# ---------------------------------------------------------------- the library's calls
def _precision(ox, kind):
    return {"fp16": ox.PRECISION_FP16, "bf16": ox.PRECISION_BF16, "fp32": ox.PRECISION_FP32}[kind]


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _block_own(s):
    import conv2d_implicit_gemm_gb300 as ox
    c, x, r, gate = s["case"], s["x"], s["residual"], s["gate"]
    t, n = c["t"], c["n"]
    total = None if r is None else torch.empty(t, n, dtype=r.dtype, device=x.device)
    y = torch.empty(t, n, dtype=x.dtype, device=x.device)
    ox.oidnx_block_norm(x.data_ptr(), n, _ptr(r), n, _ptr(total), n, y.data_ptr(), n, NORMS.index(c["post"]),
                        _ptr(s["post_weight"]), _ptr(s["post_bias"]), NORMS.index(c["pre"]), _ptr(s["pre_weight"]),
                        _ptr(s["pre_bias"]), EPS, _ptr(gate), n if c["gate"] == "groups" else 0,
                        GATES.index(c["gate_act"]), _ptr(s["scale"]), n, _ptr(s["shift"]), n, 0, c["per"],
                        (t + c["per"] - 1) // c["per"], c["alpha"], c["beta"], t, n, _precision(ox, c["type"]),
                        _precision(ox, c["stream"]), torch.cuda.current_stream().cuda_stream)
    return y if total is None else (total, y)


def _axes_own(s):
    import conv2d_implicit_gemm_gb300 as ox
    c, x = s["case"], s["qkv"]
    t, hq, hk, d = x.shape[0], c["hq"], c["hk"], c["d"]
    q_out = torch.empty(t, hq, d, dtype=x.dtype, device=x.device)
    if c["cache"]:
        k_out, v_out, slots, rows = s["k_cache"], s["v_cache"], s["slots"].data_ptr(), c["cache"]
    else:
        k_out, v_out = (torch.empty(t, hk, d, dtype=x.dtype, device=x.device) for _ in range(2))
        slots, rows = 0, t
    row, base, size = (hq + 2 * hk) * d, x.data_ptr(), x.element_size()
    ox.oidnx_qk_norm_rope_axes(base, row, d, q_out.data_ptr(), hq * d, d,
                               base + hq * d * size, row, d, k_out.data_ptr(), hk * d, d,
                               base + (hq + hk) * d * size, row, d, v_out.data_ptr(), hk * d, d,
                               int(c["norm"]), _ptr(s["q_weight"]), _ptr(s["k_weight"]), EPS, s["cos"].data_ptr(),
                               s["sin"].data_ptr(), s["cos"].shape[0], s["positions"].data_ptr(), t,
                               s["positions"].shape[0], s["pair_axes"], slots, rows, t, hq, hk, d,
                               2 * len(s["pair_axes"]), int(c["interleaved"]), _precision(ox, c["type"]),
                               torch.cuda.current_stream().cuda_stream)
    return q_out, k_out, v_out


def _cross_own(s):
    import conv2d_implicit_gemm_gb300 as ox
    c, q, k, v, mask = s["case"], s["q"], s["k"], s["v"], s["mask"]
    o = torch.empty_like(q)
    lse = torch.empty(c["b"], c["hq"], c["tq"], dtype=torch.float32, device=q.device)
    ox.oidnx_cross_attention(q.data_ptr(), *q.stride()[:3], k.data_ptr(), *k.stride()[:3], v.data_ptr(),
                             *v.stride()[:3], o.data_ptr(), *o.stride()[:3], lse.data_ptr(), _ptr(s["q_lens"]),
                             _ptr(s["kv_lens"]), _ptr(mask), c["kv"], c["b"], c["tq"], c["kv"], c["hq"], c["hk"],
                             c["d"], s["factor"], _precision(ox, c["type"]), torch.cuda.current_stream().cuda_stream)
    return o, lse


# ---------------------------------------------------------------- plain forms
def _norm(x, norm, weight, bias):
    if norm == "none":
        return x
    if norm == "layer":
        x = x - x.mean(-1, keepdim=True)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    return y if bias is None else y + bias.float()


def _block_plain(s):
    c, x = s["case"], s["x"]
    group = torch.arange(c["t"], device=x.device) // c["per"]
    branch = _norm(x.float(), c["post"], s["post_weight"], s["post_bias"]) * c["beta"]
    if s["gate"] is not None:
        gate = s["gate"].float()
        gate = torch.tanh(gate) if c["gate_act"] == "tanh" else 1 / (1 + torch.exp(-gate)) if c["gate_act"] == "sigmoid" else gate
        branch = branch * (gate if c["gate"] == "channel" else gate[group])
    total = branch if s["residual"] is None else s["residual"].float() * c["alpha"] + branch
    y = _norm(total, c["pre"], s["pre_weight"], s["pre_bias"])
    if c["modulate"]:
        y = y * (1 + s["scale"].float()[group]) + s["shift"].float()[group]
    y = y.to(x.dtype)
    return y if s["residual"] is None else (total.to(s["residual"].dtype), y)


def _head_plain(s, x, weight, cos, sin):
    c, x = s["case"], x.float()
    rot = 2 * cos.shape[-1]
    if c["norm"]:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    if weight is not None:
        x = x * weight.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["interleaved"] else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((u, w), -1).flatten(-2) if c["interleaved"] else torch.cat((u, w), -1)
    return torch.cat((turned, x[..., rot:]), -1).to(s["qkv"].dtype)


def _axes_plain(s):
    c, x = s["case"], s["qkv"]
    hq, hk = c["hq"], c["hk"]
    axis = torch.tensor(list(s["pair_axes"]), device=x.device, dtype=torch.long)
    at = s["positions"].long()[axis].t()  # [t][pairs]
    pair = torch.arange(axis.numel(), device=x.device)
    cos, sin = s["cos"][at, pair][:, None], s["sin"][at, pair][:, None]
    q = _head_plain(s, x[:, :hq], s["q_weight"], cos, sin)
    k = _head_plain(s, x[:, hq:hq + hk], s["k_weight"], cos, sin)
    v = x[:, hq + hk:].clone()
    if c["cache"]:
        to = s["slots"].long()
        s["k_cache"][to] = k
        s["v_cache"][to] = v
        return q, s["k_cache"], s["v_cache"]
    return q, k, v


def _cross_plain(s):
    c, q = s["case"], s["q"]
    b, tq, kv, hq, hk, d = (c[x] for x in ("b", "tq", "kv", "hq", "hk", "d"))
    key, row = torch.arange(kv, device=q.device)[None], torch.arange(tq, device=q.device)[None]
    held = key < (kv if s["kv_lens"] is None else s["kv_lens"].long()[:, None])
    if s["mask"] is not None:
        held = held & (s["mask"] != 0)
    held = held.expand(b, kv)
    asks = (row < (tq if s["q_lens"] is None else s["q_lens"].long()[:, None])).expand(b, tq)
    k = torch.where(held[:, :, None, None], s["k"].float(), 0.0).permute(0, 2, 3, 1)[:, :, None]
    v = torch.where(held[:, :, None, None], s["v"].float(), 0.0).permute(0, 2, 1, 3)[:, :, None]
    qg = q.float().view(b, tq, hk, hq // hk, d).permute(0, 2, 3, 1, 4)
    score = torch.matmul(qg, k) * s["factor"]
    score = score.masked_fill(~(asks[:, None, None, :, None] & held[:, None, None, None, :]), float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(total > 0, total, 1.0)
    lse = torch.where(total > 0, top + torch.log(total), float("-inf"))
    return o.permute(0, 3, 1, 2, 4).reshape(b, tq, hq, d).to(q.dtype), lse.reshape(b, hq, tq)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    size = 4 if case["type"] == "fp32" else 2
    if case["op"] == "block":
        t, n, held = case["t"], case["n"], 4 if case["stream"] == "fp32" else 2
        groups = (t + case["per"] - 1) // case["per"]
        vectors = sum((1 + case["bias"]) for x in ("post", "pre") if case[x] != "none")
        vectors += {"none": 0, "channel": 1, "groups": groups}[case["gate"]] + (2 * groups if case["modulate"] else 0)
        return {"bytes": t * n * (2 * size + (2 * held if case["residual"] else 0)) + size * n * vectors,
                "flops": 14.0 * t * n}
    if case["op"] == "axes":
        t = case["frames"] * case["rows"] * case["cols"]
        heads, d, sections = case["hq"] + 2 * case["hk"], case["d"], _sections(case)
        rows = (case["frames"], case["rows"], case["cols"], 1)  # of the table, by axis
        table = sum(8 * p * r for p, r in zip(sections, rows))
        return {"bytes": 2 * size * t * heads * d + table + 4 * t * (len(sections) + (1 if case["cache"] else 0)),
                "flops": 4.0 * t * (case["hq"] + case["hk"]) * (d + 2 * sum(sections))}
    b, tq, hq, hk, d = (case[x] for x in ("b", "tq", "hq", "hk", "d"))
    keys = [len(x) for x in _seen(case)]
    asked = [q for q, _ in _lengths(case)]
    pairs = sum(q * n for q, n in zip(asked, keys))
    moved = 2 * hk * sum(keys) + hq * sum(asked) + hq * b * tq  # keys and values, queries, output
    return {"bytes": d * size * moved + 4 * b * tq * hq + (b * case["kv"] if case["mask"] else 0),
            "flops": 4.0 * d * hq * pairs}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"block": _block_exact, "axes": _axes_exact, "cross": _cross_exact}[case["op"]](s)


def _normed(x, norm, weight, bias):
    if norm != "none":
        mean = x.sum(-1, keepdim=True) / x.shape[-1] if norm == "layer" else 0.0
        power = ((x - mean) ** 2).sum(-1, keepdim=True) / x.shape[-1]
        x = (x - mean) * (power + EPS).rsqrt() * weight.double()
        x = x + bias.double() if bias is not None else x
    return x


def _block_exact(s):
    c, totals, ys = s["case"], [], []
    act = {"plain": lambda z: z, "tanh": torch.tanh, "sigmoid": torch.sigmoid}[c["gate_act"]]
    for i in range(0, c["t"], c["per"]):  # the tokens of one group
        at = slice(i, min(i + c["per"], c["t"]))
        g = i // c["per"]
        z = _normed(s["x"][at].double(), c["post"], s["post_weight"], s["post_bias"])
        if s["gate"] is not None:
            z = z * act(s["gate"][g if c["gate"] == "groups" else 0].double())
        z = z * c["beta"]
        if s["residual"] is not None:
            z = torch.add(z, s["residual"][at].double(), alpha=c["alpha"])
            totals.append(z)
        z = _normed(z, c["pre"], s["pre_weight"], s["pre_bias"])
        if c["modulate"]:
            z = torch.addcmul(s["shift"][g].double(), z, s["scale"][g].double() + 1.0)
        ys.append(z)
    return (torch.cat(totals), torch.cat(ys)) if totals else torch.cat(ys)


def _axes_exact(s):
    c = s["case"]
    hq, hk, d = c["hq"], c["hk"], c["d"]
    x, axes = s["qkv"].double(), _pair_axes(c)
    pairs = len(axes)

    def head(z, weight):
        y = z * ((z * z).sum(-1, keepdim=True) / d + EPS).rsqrt() if c["norm"] else z.clone()
        if weight is not None:
            y = y * weight.double()
        out = y.clone()
        for r, axis in enumerate(axes):
            i, j = (2 * r, 2 * r + 1) if c["interleaved"] else (r, r + pairs)
            row = s["positions"][axis].long()
            turn = torch.complex(s["cos"][row, r].double(), s["sin"][row, r].double())[:, None]
            turned = torch.complex(y[..., i].contiguous(), y[..., j].contiguous()) * turn
            out[..., i], out[..., j] = turned.real, turned.imag
        return out

    q, k, v = head(x[:, :hq], s["q_weight"]), head(x[:, hq:hq + hk], s["k_weight"]), x[:, hq + hk:]
    if not c["cache"]:
        return q, k, v
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    kc.index_copy_(0, s["slots"].long(), k)
    vc.index_copy_(0, s["slots"].long(), v)
    return q, kc, vc


def _cross_exact(s):
    c, q = s["case"], s["q"]
    hq, hk = c["hq"], c["hk"]
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full((c["b"], hq, c["tq"]), float("-inf"), dtype=torch.float64, device=q.device)
    for i, ((nq, _), keys) in enumerate(zip(_lengths(c), _seen(c))):
        if not keys:
            continue
        at = torch.tensor(keys, device=q.device)
        k, v = (s[x][i].index_select(0, at).double().repeat_interleave(hq // hk, 1) for x in ("k", "v"))
        step = max(1, 60_000_000 // (hq * len(keys)))
        for j in range(0, nq, step):
            rows = slice(j, min(nq, j + step))
            z = torch.einsum("ihd,jhd->hij", q[i, rows].double(), k) * s["factor"]
            l = torch.logsumexp(z, -1)
            lse[i, :, rows] = l
            o[i, rows] = torch.einsum("hij,jhd->ihd", torch.exp(z - l[..., None]), v)
    return o, lse
