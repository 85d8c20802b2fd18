"""The token operators' workloads: the linear layer with its epilogue, the norm and rotation of queries and keys with
the cache append, and attention with a sliding window and sinks.  Each case is one operator at one size; run() makes
the pass with the library's calls (own) or in plain torch operations in 32 bits."""

import math

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def listed():
    return [
        # one token of a stream through a square projection with its residual: latency and the weight's bytes
        dict(name="linear_token", op="linear", m=1, n=4096, k=4096, act="none", bias=True, residual=True, type="bf16"),
        # a few streams served together, sizes that no tile divides
        dict(name="linear_few", op="linear", m=13, n=5000, k=2056, act="silu", bias=False, residual=False, type="fp16"),
        # the tokens of a frame's bottleneck map (1920x1080 / 32: 60 x 34) with an odd channel count
        dict(name="linear_odd", op="linear", m=2040, n=1001, k=999, act="gelu", bias=True, residual=True, type="fp16"),
        # a long prompt through the widening projection of a block
        dict(name="linear_prompt", op="linear", m=8192, n=8192, k=4096, act="gelu_tanh", bias=True, residual=False,
             type="bf16"),
        # one new token of one stream: the smallest call of all
        dict(name="norm_token", op="norm", t=1, hq=32, hk=8, d=128, rot=128, interleaved=False, weight=True, cache=512,
             type="bf16"),
        # a map's tokens, part of each head rotated in adjacent pairs
        dict(name="norm_odd", op="norm", t=2040, hq=7, hk=7, d=72, rot=40, interleaved=True, weight=False, cache=0,
             type="fp16"),
        # a long prompt, keys and values appended to the cache
        dict(name="norm_prompt", op="norm", t=16384, hq=32, hk=8, d=128, rot=128, interleaved=False, weight=True,
             cache=20000, type="bf16"),
        # one token of one endless stream over its ring cache
        dict(name="attn_token", op="attn", b=1, tq=1, kv=100000, cap=4100, hq=32, hk=8, d=128, window=4096, sinks=4,
             ragged=False, type="bf16"),
        # one token each of many streams of all lengths
        dict(name="attn_tokens", op="attn", b=64, tq=1, kv=8191, cap=8192, hq=32, hk=8, d=128, window=4096, sinks=4,
             ragged=True, type="bf16"),
        # prompts of different lengths, some longer than what is held, heads that fill no tile
        dict(name="attn_ragged", op="attn", b=5, tq=700, kv=1501, cap=1600, hq=6, hk=2, d=80, window=333, sinks=3,
             ragged=True, type="fp16"),
        # small heads, no window
        dict(name="attn_causal", op="attn", b=2, tq=4096, kv=4096, cap=4096, hq=8, hk=8, d=64, window=0, sinks=0,
             ragged=False, type="fp16"),
        # a long prompt through a sliding window with sinks
        dict(name="attn_prompt", op="attn", b=1, tq=8192, kv=8192, cap=8192, hq=16, hk=4, d=128, window=2048, sinks=4,
             ragged=False, type="bf16"),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("linear", "norm", "attn"))
    kind = rng.choice(("fp16", "bf16"))
    if op == "linear":
        m = rng.choice((1, _log(rng, 1, 64), _log(rng, 64, 8192)))
        n, k = _log(rng, 256, 8192), _log(rng, 256, 8192)
        if rng.random() < 0.7:  # the usual widths; the others stay odd
            n, k = (n + 7) // 8 * 8, (k + 7) // 8 * 8
        if m * n * k > 8192 * 8192 * 4096:
            k = 4096
        return dict(op=op, m=m, n=n, k=k, act=rng.choice(ACTS), bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                    type=kind)
    if op == "norm":
        d = rng.choice((64, 128, 128, 8 * rng.randint(4, 32)))
        hk = rng.randint(1, 8)
        hq = hk * rng.choice((1, 2, 4))
        t = rng.choice((1, _log(rng, 1, 64), _log(rng, 64, 16384)))
        kind = rng.choice(("fp16", "bf16", "fp32"))
        t = min(t, 200_000_000 // (d * (hq + 2 * hk) * (4 if kind == "fp32" else 2)))
        return dict(op=op, t=t, hq=hq, hk=hk, d=d, rot=rng.choice((d, d // 2)), interleaved=rng.random() < 0.5,
                    weight=rng.random() < 0.7, cache=rng.choice((0, t + rng.randint(0, 512))),
                    type=kind)
    d = rng.choice((64, 128, 128, 8 * rng.randint(4, 16)))
    hk = rng.randint(1, 8)
    sinks = rng.choice((0, 4, rng.randint(1, 40)))
    if rng.random() < 0.5:  # tokens
        b, window = _log(rng, 1, 64), rng.choice((0, _log(rng, 64, 8192)))
        kv = _log(rng, 64, min(32768, 380_000_000 // (b * hk * d * 2)))
        cap = min(kv + 1, window + sinks + 3) if window and rng.random() < 0.5 else kv + rng.randint(0, 300)
        return dict(op=op, b=b, tq=rng.choice((1, 1, 1, rng.randint(2, 8))), kv=kv, cap=cap, hq=hk * rng.choice((1, 2, 4, 8)),
                    hk=hk, d=d, window=window, sinks=min(sinks, cap - 1), ragged=rng.random() < 0.5, type=kind)
    hk, group = rng.randint(1, 4), rng.choice((1, 2, 4))
    tq = _log(rng, 16, 8192 if hk * group <= 8 else 4096)
    kv = tq + rng.choice((0, 0, _log(rng, 1, 2048)))
    b = max(1, min(4, 8192 // kv))
    return dict(op=op, b=b, tq=tq, kv=kv, cap=kv + rng.choice((0, rng.randint(0, 100))), hq=hk * group,
                hk=hk, d=d, window=rng.choice((0, _log(rng, 16, 4096))), sinks=min(sinks, kv), ragged=rng.random() < 0.5,
                type=kind)


def _lengths(case):
    """(query length, key length) of each sequence; ragged batches hold short and empty ones among the full."""
    b, tq, kv = case["b"], case["tq"], case["kv"]
    if not case["ragged"]:
        return [(tq, kv)] * b
    got = []
    for i in range(b):
        part = ((i * 37 + 11) % 64) / 64.0
        n = kv if i == 0 else 0 if i == 3 else max(1, int(kv * part))
        q = tq if i % 2 == 0 else max(1, (tq * 5) // 7)
        got.append((q, n))
    return got


def _held(case, n):
    """(slots, positions) that a cache holds after n keys, as lists of ranges: the sinks, then the ring."""
    cap, sinks = case["cap"], case["sinks"]
    first = min(n, sinks)
    return first, max(sinks, n - (cap - sinks)) if n > first else first


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind = TYPES[case["type"]]

    def normal(*shape, scale=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale + mean).to(kind)

    s = {"case": dict(case)}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        s["x"] = normal(m, k)
        s["w"] = normal(n, k, scale=1 / math.sqrt(k))
        s["bias"] = normal(n, scale=0.5) if case["bias"] else None
        s["residual"] = normal(m, n) if case["residual"] else None
    elif case["op"] == "norm":
        t, hq, hk, d, rot = (case[x] for x in ("t", "hq", "hk", "d", "rot"))
        s["qkv"] = normal(t, hq + 2 * hk, d, scale=1.5)  # as one projection wrote them
        s["q_weight"] = normal(d, scale=0.2, mean=1.0) if case["weight"] else None
        s["k_weight"] = normal(d, scale=0.2, mean=1.0) if case["weight"] else None
        rows = max(t, case["cache"]) + 64
        angle = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * (
            10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot))
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        begin = int(torch.randint(0, 64, (1,), generator=g, device="cuda").item())
        s["positions"] = torch.arange(begin, begin + t, device="cuda", dtype=torch.int32)
        if case["cache"]:
            s["slots"] = ((torch.arange(t, device="cuda") + begin) % case["cache"]).to(torch.int32)
            s["k_cache"], s["v_cache"] = normal(case["cache"], hk, d), normal(case["cache"], hk, d)
    else:
        b, tq, cap, hq, hk, d = (case[x] for x in ("b", "tq", "cap", "hq", "hk", "d"))
        s["q"] = normal(b, tq, hq, d, scale=1.2)
        s["k"], s["v"] = normal(b, cap, hk, d, scale=1.2), normal(b, cap, hk, d)
        lengths = _lengths(case)
        for i, (_, n) in enumerate(lengths):  # slots that no key was written to hold anything
            s["k"][i, min(n, cap):] = float("nan")
            s["v"][i, min(n, cap):] = float("nan")
        s["q_lens"] = torch.tensor([q for q, _ in lengths], dtype=torch.int32, device="cuda")
        s["kv_lens"] = torch.tensor([n for _, n in lengths], dtype=torch.int32, device="cuda")
        s["scale"] = 1 / math.sqrt(d)
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return {"linear": _linear_own, "norm": _norm_own, "attn": _attn_own}[op](s)
    return {"linear": _linear_plain, "norm": _norm_plain, "attn": _attn_plain}[op](s)


# ---------------------------------------------------------------- the library's calls
def _precision(ox, t):
    return {torch.float16: ox.PRECISION_FP16, torch.bfloat16: ox.PRECISION_BF16, torch.float32: ox.PRECISION_FP32}[t.dtype]


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _linear_own(s):
    import conv2d_implicit_gemm_gb300 as ox
    c, x, w, r = s["case"], s["x"], s["w"], s["residual"]
    y = torch.empty(c["m"], c["n"], dtype=x.dtype, device=x.device)
    ox.oidnx_linear(x.data_ptr(), c["k"], w.data_ptr(), c["k"], _ptr(s["bias"]), _ptr(r), c["n"], y.data_ptr(), c["n"],
                    c["m"], c["n"], c["k"], ACTS.index(c["act"]), _precision(ox, x),
                    torch.cuda.current_stream().cuda_stream)
    return y


def _norm_own(s):
    import conv2d_implicit_gemm_gb300 as ox
    c, x = s["case"], s["qkv"]
    t, hq, hk, d = c["t"], c["hq"], c["hk"], c["d"]
    q_out = torch.empty(t, hq, d, dtype=x.dtype, device=x.device)
    if c["cache"]:
        k_out, v_out, slots, rows = s["k_cache"], s["v_cache"], s["slots"].data_ptr(), c["cache"]
    else:
        k_out, v_out = (torch.empty(t, hk, d, dtype=x.dtype, device=x.device) for _ in range(2))
        slots, rows = 0, t
    row, base, size = (hq + 2 * hk) * d, x.data_ptr(), x.element_size()
    ox.oidnx_qk_norm_rope(base, row, d, q_out.data_ptr(), hq * d, d,
                          base + hq * d * size, row, d, k_out.data_ptr(), hk * d, d,
                          base + (hq + hk) * d * size, row, d, v_out.data_ptr(), hk * d, d,
                          _ptr(s["q_weight"]), _ptr(s["k_weight"]), 1e-6, s["cos"].data_ptr(), s["sin"].data_ptr(),
                          s["cos"].shape[0], s["positions"].data_ptr(), slots, rows, t, hq, hk, d, c["rot"],
                          int(c["interleaved"]), _precision(ox, x), torch.cuda.current_stream().cuda_stream)
    return q_out, k_out, v_out


def _attn_own(s):
    import conv2d_implicit_gemm_gb300 as ox
    c, q, k, v = s["case"], s["q"], s["k"], s["v"]
    o = torch.empty_like(q)
    lse = torch.empty(c["b"], c["hq"], c["tq"], dtype=torch.float32, device=q.device)
    ox.oidnx_window_attention(q.data_ptr(), *q.stride()[:3], k.data_ptr(), *k.stride()[:3], v.data_ptr(),
                              *v.stride()[:3], o.data_ptr(), *o.stride()[:3], lse.data_ptr(), s["q_lens"].data_ptr(),
                              s["kv_lens"].data_ptr(), c["b"], c["tq"], c["cap"], c["hq"], c["hk"], c["d"],
                              c["window"], c["sinks"], s["scale"], _precision(ox, q),
                              torch.cuda.current_stream().cuda_stream)
    return o, lse


# ---------------------------------------------------------------- plain forms
def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _linear_plain(s):
    z = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    z = _act(z, s["case"]["act"])
    if s["residual"] is not None:
        z = z + s["residual"].float()
    return z.to(s["x"].dtype)


def _norm_rotate(x, weight, cos, sin, rot, interleaved):
    x = x.float()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    if weight is not None:
        y = y * weight.float()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((turned, y[..., rot:]), -1)


def _norm_plain(s):
    c, x = s["case"], s["qkv"]
    hq, hk = c["hq"], c["hk"]
    at = s["positions"].long()
    cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
    q = _norm_rotate(x[:, :hq], s["q_weight"], cos, sin, c["rot"], c["interleaved"]).to(x.dtype)
    k = _norm_rotate(x[:, hq:hq + hk], s["k_weight"], cos, sin, c["rot"], c["interleaved"]).to(x.dtype)
    v = x[:, hq + hk:].clone()
    if c["cache"]:
        to = s["slots"].long()
        s["k_cache"][to] = k
        s["v_cache"][to] = v
        return q, s["k_cache"], s["v_cache"]
    return q, k, v


def _attn_plain(s):
    c, q = s["case"], s["q"]
    b, tq, cap, hq, hk, d, window, sinks = (c[x] for x in ("b", "tq", "cap", "hq", "hk", "d", "window", "sinks"))
    slot = torch.arange(cap, device=q.device)
    n = s["kv_lens"].long()[:, None]
    # the position whose key a slot holds: the last one before n that falls on it; -1: none
    ring = max(cap - sinks, 1)
    last = n - 1 - (n - 1 - slot) % ring
    where = torch.where(slot < sinks, slot, torch.where(last >= sinks, last, -1))
    where = torch.where((where < n) & (where >= 0), where, -1)
    row = torch.arange(tq, device=q.device)
    p = torch.where(row < s["q_lens"].long()[:, None], row + n - s["q_lens"].long()[:, None], -1)
    j, p = where[:, None, :], p[:, :, None]
    seen = (j >= 0) & (j <= p)
    if window:
        seen = seen & ((j > p - window) | (j < sinks))
    held = (where >= 0)[:, :, None, None]
    k = torch.where(held, s["k"].float(), 0.0).permute(0, 2, 3, 1)[:, :, None]
    v = torch.where(held, s["v"].float(), 0.0).permute(0, 2, 1, 3)[:, :, None]
    qg = q.float().view(b, tq, hk, hq // hk, d).permute(0, 2, 3, 1, 4)
    score = torch.matmul(qg, k) * s["scale"]
    score = score.masked_fill(~seen[:, None, None], float("-inf"))
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
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": size * (m * k + n * k + m * n + (n if case["bias"] else 0) + (m * n if case["residual"] else 0)),
                "flops": 2.0 * m * n * k}
    if case["op"] == "norm":
        t, heads, d = case["t"], case["hq"] + 2 * case["hk"], case["d"]
        return {"bytes": 2 * size * t * heads * d + 4 * t * case["rot"] + 8 * t,
                "flops": 8.0 * t * (case["hq"] + case["hk"]) * d}
    d, hq, hk, window, sinks = (case[x] for x in ("d", "hq", "hk", "window", "sinks"))
    moved, pairs = 0, 0
    for q, n in _lengths(case):
        first, begin = _held(case, n)
        top = min(first, n)
        low_seen = n
        for i in range(q):
            p = n - q + i
            if p < 0:
                continue
            low = max(begin, p - window + 1) if window else begin
            pairs += min(top, p + 1) + max(0, p + 1 - max(low, top))
            low_seen = min(low_seen, max(low, top))
        moved += 2 * (top + max(0, n - low_seen)) * hk * d * size
    b, tq = case["b"], case["tq"]
    return {"bytes": moved + 2 * b * tq * hq * d * size + 4 * b * tq * hq, "flops": 4.0 * d * hq * pairs}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _linear_exact, "norm": _norm_exact, "attn": _attn_exact}[case["op"]](s)


def _linear_exact(s):
    c, got = s["case"], []
    w = s["w"].double()
    for x, r in zip(s["x"].split(1024), (s["residual"] if s["residual"] is not None else s["x"]).split(1024)):
        z = torch.einsum("ik,jk->ij", x.double(), w)
        if c["bias"]:
            z += s["bias"].double()
        if c["act"] == "relu":
            z = torch.where(z > 0, z, torch.zeros_like(z))
        elif c["act"] == "gelu":
            z = z * torch.special.ndtr(z)
        elif c["act"] == "gelu_tanh":
            z = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        elif c["act"] == "silu":
            z = z * torch.sigmoid(z)
        got.append(z + r.double() if c["residual"] else z)
    return torch.cat(got)


def _norm_exact(s):
    c = s["case"]
    hq, hk, d, rot = c["hq"], c["hk"], c["d"], c["rot"]
    x = s["qkv"].double()
    first = torch.arange(rot // 2, device=x.device) * (2 if c["interleaved"] else 1)
    second = first + (1 if c["interleaved"] else rot // 2)
    turn = torch.complex(s["cos"].double(), s["sin"].double())[s["positions"].long()][:, None]

    def head(z, weight):
        y = z * (z.pow(2).sum(-1, keepdim=True) / d + 1e-6).rsqrt()
        if weight is not None:
            y = y * weight.double()
        r = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
        out = y.clone()
        out[..., first], out[..., second] = r.real, r.imag
        return out

    q, k, v = head(x[:, :hq], s["q_weight"]), head(x[:, hq:hq + hk], s["k_weight"]), x[:, hq + hk:]
    if not c["cache"]:
        return q, k, v
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    kc.index_copy_(0, s["slots"].long(), k)
    vc.index_copy_(0, s["slots"].long(), v)
    return q, kc, vc


def _attn_exact(s):
    c, q = s["case"], s["q"]
    cap, hq, hk, d, window, sinks = (c[x] for x in ("cap", "hq", "hk", "d", "window", "sinks"))
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full((c["b"], hq, c["tq"]), float("-inf"), dtype=torch.float64, device=q.device)
    for i, (nq, n) in enumerate(_lengths(c)):
        if n == 0:
            continue
        first, begin = _held(c, n)
        keys = torch.tensor(list(range(first)) + list(range(max(begin, first), n)), device=q.device)
        slots = torch.where(keys < sinks, keys, sinks + (keys - sinks) % max(cap - sinks, 1))
        k, v = s["k"][i].index_select(0, slots).double(), s["v"][i].index_select(0, slots).double()
        for at in range(0, nq, 1024):
            rows = torch.arange(at, min(nq, at + 1024), device=q.device)
            p = (n - nq + rows)[:, None]
            hidden = keys[None] > p
            if window:
                hidden = hidden | ((keys[None] <= p - window) & (keys[None] >= sinks))
            some = ~hidden.all(1)
            for h in range(hq):
                z = q[i, rows, h].double() @ k[:, h // (hq // hk)].t() * s["scale"]
                z[hidden] = float("-inf")
                l = torch.logsumexp(z, 1)
                lse[i, h, rows] = l
                w = torch.exp(z[some] - l[some, None])
                o[i, rows[some], h] = w @ v[:, h // (hq // hk)]
    return o, lse
