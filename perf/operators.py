"""The measured cases of the operators around the quantized linears: the 4-bit
paged KV cache (page assignment, append, read-back, attention) and the fused
residual norms.  `run` computes each in plain torch, or with `own` through the
package's entry points."""
import math

import torch

own = False

HALF_MAX = 65504.0


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step of a small batch: the page table and slot of each new token
        {"name": "assign_decode_64", "op": "assign", "requests": 64, "new": 1, "context": 4096, "page": 64},
        # a wave of prompts of different lengths joining running requests, small pages
        {"name": "assign_prompts_256", "op": "assign", "requests": 256, "new": 509, "context": 8192, "page": 16},
        # one decode step's keys and values of Llama-3.1-8B's heads
        {"name": "append_decode_32", "op": "append", "tokens": 32, "q_heads": 32, "kv_heads": 8, "head_dim": 128,
         "rotary": 128, "page": 64},
        # a chunk of prompts at Llama-3.1-70B's heads, an odd number of tokens
        {"name": "append_prompt_4099", "op": "append", "tokens": 4099, "q_heads": 64, "kv_heads": 8, "head_dim": 128,
         "rotary": 128, "page": 16},
        # the norm before a linear for one token
        {"name": "norm_quant_1", "op": "norm", "tokens": 1, "width": 4096, "post": False, "gate": "none",
         "residual": "float16", "quantize": True},
        # sandwich norms with a gate per channel and a 32-bit residual stream, fp16 out
        {"name": "norm_post_1024", "op": "norm", "tokens": 1024, "width": 8192, "post": True, "gate": "channel",
         "residual": "float32", "quantize": False},
        # a prompt chunk at the 8B width, gated per token and channel, codes for the next linear
        {"name": "norm_quant_2047", "op": "norm", "tokens": 2047, "width": 4096, "post": False, "gate": "token",
         "residual": "float16", "quantize": True},
        # one request's decode step at a short context: latency
        {"name": "attend_decode_1", "op": "attend", "requests": 1, "query": 1, "short": 1003, "long": 1003,
         "q_heads": 32, "kv_heads": 8, "head_dim": 128, "page": 16},
        # a batch of requests of very different lengths, one token each
        {"name": "attend_decode_64", "op": "attend", "requests": 64, "query": 1, "short": 100, "long": 8100,
         "q_heads": 32, "kv_heads": 8, "head_dim": 128, "page": 64},
        # few requests with very long contexts at Llama-3.1-70B's heads
        {"name": "attend_decode_long", "op": "attend", "requests": 4, "query": 1, "short": 100000, "long": 131071,
         "q_heads": 64, "kv_heads": 8, "head_dim": 128, "page": 128},
        # a few proposed tokens per request checked at once, heads of 64
        {"name": "attend_verify_16", "op": "attend", "requests": 16, "query": 3, "short": 700, "long": 5001,
         "q_heads": 16, "kv_heads": 4, "head_dim": 64, "page": 32},
        # chunks of prompts behind cached prefixes
        {"name": "attend_prompt_1024", "op": "attend", "requests": 2, "query": 1024, "short": 5000, "long": 8192,
         "q_heads": 32, "kv_heads": 8, "head_dim": 128, "page": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["assign", "append", "norm", "attend", "attend", "attend"])
    page = rng.choice([16, 32, 64, 128])
    heads = rng.choice([(32, 8, 128), (64, 8, 128), (16, 16, 64), (8, 1, 128), (24, 8, 128), (16, 2, 64)])
    if op == "assign":
        new = rng.choice([1, 1, _log(rng, 2, 512)])
        return {"op": op, "requests": _log(rng, 1, max(2, min(2048, 130000 // new))), "new": new,
                "context": _log(rng, 1, 8192), "page": page}
    if op == "append":
        return {"op": op, "tokens": _log(rng, 1, 4096), "q_heads": heads[0], "kv_heads": heads[1],
                "head_dim": heads[2], "rotary": rng.choice([heads[2], heads[2] // 2]), "page": page}
    if op == "norm":
        width = 128 * _log(rng, 4, 64)
        return {"op": op, "tokens": _log(rng, 1, min(2048, 7000000 // width)), "width": width,
                "post": rng.random() < 0.5, "gate": rng.choice(["none", "channel", "token"]),
                "residual": rng.choice(["float16", "float32"]), "quantize": rng.random() < 0.5}
    if rng.random() < 0.7:  # decode and checks of a few proposed tokens
        requests = _log(rng, 1, 128)
        query = rng.choice([1, 1, 2, 3, 5])
        long = max(query, _log(rng, 16, min(131072, 430000 // requests)))
    else:  # chunks of prompts
        requests = rng.choice([1, 1, 2, 3, 4])
        query = _log(rng, 8, 36864 // heads[0] // requests)
        long = query + _log(rng, 1, 8192)
    return {"op": op, "requests": requests, "query": query, "short": max(query, long // rng.choice([1, 2, 7])),
            "long": long, "q_heads": heads[0], "kv_heads": heads[1], "head_dim": heads[2], "page": page}


def _spread(n, lo, hi):
    """n whole numbers in [lo, hi], unevenly spread, the first one hi."""
    return [hi - int((hi - lo) * (i * 0.6180339887498949 % 1.0)) for i in range(n)]


def _lengths(case):
    """Cached tokens of each request (its new ones among them) and its queries."""
    kv = _spread(case["requests"], case["short"], case["long"])
    if case["query"] <= 8:
        return kv, [case["query"]] * case["requests"]
    return kv, [min(k, q) for k, q in zip(kv, _spread(case["requests"], case["query"] * 3 // 4, case["query"]))]


def work(case):
    if case["op"] == "assign":
        B = case["requests"]
        new, ctx = _spread(B, (case["new"] + 1) // 2, case["new"]), _spread(B, 0, case["context"])
        p = case["page"]
        entries = sum(-(-(c + n) // p) - c // p for c, n in zip(ctx, new))
        return {"bytes": 8 * B + 8 * B + 4 + 12 * B * case["new"] + 8 * entries, "flops": 0}
    if case["op"] == "append":
        T, D = case["tokens"], case["head_dim"]
        q, kv = case["q_heads"] * D, case["kv_heads"] * D
        rope = 4 * case["rotary"] + 12
        # the cache is written and read back once (codes and scales), and its values written in fp16
        return {"bytes": T * (2 * (q + 2 * kv) + rope + 2 * q + 2 * (kv + 8 * case["kv_heads"]) + 4 * kv),
                "flops": T * (3 * (q + kv) + 6 * kv)}
    if case["op"] == "norm":
        n, K = case["tokens"] * case["width"], case["width"]
        r = 2 if case["residual"] == "float16" else 4
        per = 2 + 2 * r + {"none": 0, "channel": 0, "token": 2}[case["gate"]]
        # fp16 out, or codes and scales out, read back once, and their values in fp16
        per += 2 if not case["quantize"] else 2 * (1 + 4 / 128) + 2
        weights = 2 * K * (1 + case["post"] + (case["gate"] == "channel"))
        return {"bytes": n * per + weights, "flops": 12 * n}
    kv, qs = _lengths(case)
    D, H = case["head_dim"], case["q_heads"]
    pairs = sum(q * (k - q) + q * (q + 1) // 2 for k, q in zip(kv, qs))
    cache = sum(kv) * 2 * case["kv_heads"] * (D // 2 + 4)
    return {"bytes": cache + 4 * sum(qs) * H * D + 4 * sum(-(-k // case["page"]) for k in kv),
            "flops": 4 * pairs * D * H}


# ------------------------------------------------------------------ inputs

def _rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


class _Cache:
    """The parts of a 4-bit paged cache: codes uint8 [pages, 2, heads, page,
    dim / 2] and meta int32 [pages, 2, heads, page]."""

    def __init__(self, codes, meta):
        self.codes, self.meta = codes, meta


def _cache(g, pages, heads, page, dim):
    codes = torch.randint(0, 256, (pages, 2, heads, page, dim // 2), generator=g, device="cuda", dtype=torch.uint8)
    # codes spread like those of normal values: each nibble the mean of two uniform ones
    codes = ((codes & 0x0E) + (codes >> 4 & 0x0E) >> 1) | (torch.roll(codes, 1, -1) & 0xE0) >> 1 | (codes & 0x01) << 7
    scale = (0.2 + 0.2 * torch.rand((pages, 2, heads, page), generator=g, device="cuda")).to(torch.float16)
    zero = torch.randint(5, 10, (pages, 2, heads, page), generator=g, device="cuda", dtype=torch.int32)
    return _Cache(codes, (scale.view(torch.int16).to(torch.int32) & 0xFFFF) | zero << 16)


def _handle(cache):
    from mixed_precision_quantized_act_b200 import KV4Cache
    return KV4Cache(cache.codes, cache.meta)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    p = case.get("page", 0)
    if case["op"] == "assign":
        B = case["requests"]
        new, ctx = _spread(B, (case["new"] + 1) // 2, case["new"]), _spread(B, 0, case["context"])
        W = -(-(case["context"] + case["new"]) // p)
        s["ctx"], s["new"] = _ints(ctx), _ints(new)
        pages = torch.randperm(2 * B * W, generator=g, device="cuda").to(torch.int32)
        used = torch.arange(W, device="cuda")[None, :] < (s["ctx"][:, None] + p - 1) // p
        s["table"] = torch.where(used, pages[:B * W].view(B, W), -1)
        s["free"], s["count"] = pages[B * W:].contiguous(), _ints([B * W - seed % 7 % W])
        T = B * case["new"]
        s["seq"], s["cu"] = torch.empty_like(s["ctx"]), torch.empty(B + 1, dtype=torch.int32, device="cuda")
        s["slots"] = torch.empty(T, dtype=torch.int64, device="cuda")
        s["pos"] = torch.empty(T, dtype=torch.int32, device="cuda")
        s["left"], s["status"] = torch.empty_like(s["count"]), torch.empty_like(s["count"])
    elif case["op"] == "append":
        T, D, R, H = case["tokens"], case["head_dim"], case["rotary"], case["kv_heads"]
        qkv = _rand(g, T, case["q_heads"] + 2 * H, D)
        qkv *= 1 + 7 * (torch.rand(D, generator=g, device="cuda") < 0.03)  # a few large channels, as in real keys
        s["qkv"] = qkv.to(torch.float16)
        pages = 2 * (-(-T // p)) + 1
        s["cache"] = _cache(g, pages, H, p, D)
        s["slots"] = torch.randperm(pages * p, generator=g, device="cuda")[:T].contiguous()
        far = 16384
        angle = torch.outer(torch.arange(far, dtype=torch.float64, device="cuda"),
                            500000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R))
        s["rope"] = torch.cat((angle.cos(), angle.sin()), 1).to(torch.float32)
        s["pos"] = torch.randint(0, far, (T,), generator=g, device="cuda", dtype=torch.int32)
        s["q_out"] = torch.empty((T, case["q_heads"], D), dtype=torch.float16, device="cuda")
        s["k_out"], s["v_out"] = (torch.empty((T, H, D), dtype=torch.float16, device="cuda") for _ in range(2))
    elif case["op"] == "norm":
        M, K = case["tokens"], case["width"]
        kind = getattr(torch, case["residual"])
        outlier = 1 + 19 * (torch.rand(K, generator=g, device="cuda") < 0.01)
        s["x"] = _rand(g, M, K).to(torch.float16)
        s["r"] = (_rand(g, M, K) * outlier).to(kind)
        s["w"] = (1 + 0.1 * _rand(g, K)).to(torch.float16)
        s["w_post"] = (1 + 0.1 * _rand(g, K)).to(torch.float16) if case["post"] else None
        rows = {"none": 0, "channel": 1, "token": M}[case["gate"]]
        s["gate"] = torch.sigmoid(_rand(g, rows, K)).to(torch.float16) if rows else None
        s["scale"], s["eps"] = 0.5 if case["post"] else 1.0, 1e-5
        s["r_out"] = torch.empty_like(s["r"])
        s["y"] = torch.empty_like(s["x"])
        if case["quantize"]:
            s["codes"] = torch.empty((M, K), dtype=torch.int8, device="cuda")
            s["s_a"] = torch.empty((M, K // 128), dtype=torch.float32, device="cuda")
    else:
        kv, qs = _lengths(case)
        used = [-(-k // p) for k in kv]
        W, pages = max(used), sum(used) + 3
        s["cache"] = _cache(g, pages, case["kv_heads"], p, case["head_dim"])
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        ends = _ints(used).cumsum(0)
        j = torch.arange(W, device="cuda")[None, :]
        first = (ends - _ints(used))[:, None]
        s["table"] = torch.where(j < _ints(used)[:, None], order[(first + j).clamp(max=pages - 1)], -1)
        s["kv"], s["cu"] = _ints(kv), _ints([sum(qs[:i]) for i in range(len(qs) + 1)])
        s["max_q"], s["max_kv"] = max(qs), max(kv)
        s["q"] = _rand(g, sum(qs), case["q_heads"], case["head_dim"]).to(torch.float16)
        s["out"] = torch.empty_like(s["q"])
        s["scale"] = 1.0 / math.sqrt(case["head_dim"])
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _own_assign(s):
    import mixed_precision_quantized_act_b200 as mx
    mx.kv4_assign_into(s["ctx"], s["new"], s["table"], s["free"], s["count"], s["case"]["page"], s["seq"], s["cu"],
                       s["slots"], s["pos"], s["left"], s["status"])
    return {k: s[k] for k in ("seq", "cu", "slots", "pos", "table", "left", "status")}


def _own_append(s):
    import mixed_precision_quantized_act_b200 as mx
    if "handle" not in s:
        s["handle"] = _handle(s["cache"])
    c = s["case"]
    q, k, v = s["qkv"].split((c["q_heads"], c["kv_heads"], c["kv_heads"]), 1)
    mx.kv4_append_into(k, v, s["slots"], s["handle"], q=q, q_out=s["q_out"], positions=s["pos"], rope=s["rope"])
    mx.kv4_read_into(s["slots"], s["handle"], s["k_out"], s["v_out"])
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def _own_norm(s):
    import mixed_precision_quantized_act_b200 as mx
    c = s["case"]
    more = {"x": s["x"], "r_out": s["r_out"], "w_post": s["w_post"], "gate": s["gate"], "scale": s["scale"],
            "eps": s["eps"]}
    if c["quantize"]:
        mx.residual_norm_quantize_into(s["r"], s["w"], s["codes"], s["s_a"], **more)
        mx.dequantize_act_into(s["codes"], s["s_a"], s["y"])
    else:
        mx.residual_norm_into(s["r"], s["w"], s["y"], **more)
    return {"r": s["r_out"], "y": s["y"]}


def _own_attend(s):
    import mixed_precision_quantized_act_b200 as mx
    if "handle" not in s:
        s["handle"] = _handle(s["cache"])
        s["workspace"] = mx.kv4_attention_workspace(s["case"]["requests"], s["max_q"], s["case"]["q_heads"],
                                                    s["handle"], s["table"].shape[1])
    mx.kv4_attention_into(s["q"], s["handle"], s["table"], s["kv"], s["cu"], s["max_q"], s["out"], s["workspace"],
                          scale=s["scale"])
    return {"out": s["out"]}


_own = {"assign": _own_assign, "append": _own_append, "norm": _own_norm, "attend": _own_attend}


def _plain_assign(s):
    p, T, (B, W) = s["case"]["page"], s["slots"].numel(), s["table"].shape
    ctx, new, count = s["ctx"].long(), s["new"].long(), s["count"].long()
    have, need = (ctx + p - 1) // p, (ctx + new + p - 1) // p
    off = (need - have).cumsum(0) - (need - have)
    cu = torch.cat((torch.zeros_like(count), new.cumsum(0)))
    status = ((need - have).sum() > count) * 1 + (need > W).any() * 2 + (cu[-1] > T) * 4 \
        + ((ctx < 0) | (new < 0)).any() * 8
    good = status == 0
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=B - 1)
    pos = ctx[b] + t - cu[b]
    fresh = pos // p - have[b]
    popped = s["free"][(count - 1 - off[b] - fresh).clamp(0, s["free"].numel() - 1)]
    at = torch.where(fresh < 0, s["table"][b, (pos // p).clamp(0, W - 1)], popped).long()
    here = (t < cu[-1]) & good
    j = torch.arange(W, device="cuda")[None, :]
    taken = s["free"][(count - 1 - off[:, None] - (j - have[:, None])).clamp(0, s["free"].numel() - 1)]
    table = torch.where((j >= have[:, None]) & (j < need[:, None]) & good, taken, s["table"])
    return {"seq": torch.where(good, ctx + new, ctx).int(), "cu": torch.where(good, cu, 0).int(),
            "slots": torch.where(here, at * p + pos % p, -1), "pos": torch.where(here, pos, -1).int(),
            "table": table, "left": torch.where(good, count - (need - have).sum(), count).int(),
            "status": status.int().reshape(1)}


def _rotated(x, rope, R):
    """Half-split rotation of the first R channels: fp32, rounded to fp16."""
    cos, sin = rope[:, None, :R // 2], rope[:, None, R // 2:]
    x = x.float()
    a, b = x[..., :R // 2], x[..., R // 2:R]
    return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., R:]), -1).to(torch.float16)


def _codes(x):
    """4-bit codes, fp16 scale and zero point of each row of x (fp16 values)."""
    x = x.float()
    lo, hi = x.amin(-1, keepdim=True).clamp(max=0), x.amax(-1, keepdim=True).clamp(min=0)
    scale = ((hi - lo) / torch.full_like(hi, 15)).to(torch.float16)
    step = torch.where(scale > 0, scale, 1).float()
    zero = (-lo / step).round().clamp(0, 15)
    code = ((x / step).round() + zero).clamp(0, 15)
    return torch.where(scale > 0, code, 0), scale, torch.where(scale > 0, zero, 0)


def _values(codes, meta):
    """fp32 values of cached rows: codes uint8 [..., D/2], meta int32 [...]."""
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float()
    scale = (meta & 0xFFFF).to(torch.int16).view(torch.float16).float()
    return (q - (meta >> 16 & 15).float()[..., None]) * scale[..., None]


def _plain_append(s):
    c = s["case"]
    q, k, v = s["qkv"].split((c["q_heads"], c["kv_heads"], c["kv_heads"]), 1)
    rope = s["rope"][s["pos"].long()]
    q = _rotated(q, rope, c["rotary"])
    kv = torch.stack((_rotated(k, rope, c["rotary"]), v), 1)
    code, scale, zero = _codes(kv)
    code = code.to(torch.uint8)
    page, row = s["slots"] // c["page"], s["slots"] % c["page"]
    cache = s["cache"]
    cache.codes[page, :, :, row] = code[..., 0::2] | code[..., 1::2] << 4
    cache.meta[page, :, :, row] = (scale.view(torch.int16).to(torch.int32) & 0xFFFF | zero.to(torch.int32) << 16)[..., 0]
    kept = _values(cache.codes[page, :, :, row], cache.meta[page, :, :, row]).clamp(-HALF_MAX, HALF_MAX).half()
    return {"q": q, "k": kept[:, 0], "v": kept[:, 1]}


def _plain_norm(s):
    u = s["x"].float()
    if s["w_post"] is not None:
        u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + s["eps"]) * s["w_post"].float()
    if s["gate"] is not None:
        u = u * s["gate"].float()
    r = (s["r"].float() + s["scale"] * u).to(s["r"].dtype)
    y = r.float() * torch.rsqrt(r.float().square().mean(-1, keepdim=True) + s["eps"]) * s["w"].float()
    y = y.half()
    if s["case"]["quantize"]:
        a = y.float().view(y.shape[0], -1, 128)
        s_a = a.abs().amax(-1, keepdim=True) / torch.full((1,), 127.0, device="cuda")
        codes = (a / torch.where(s_a > 0, s_a, 1)).round().clamp(-127, 127)
        y = (codes * s_a).view_as(y).half()
    return {"r": r, "y": y}


def _plain_attend(s):
    c = s["case"]
    B, Hq, H, D, Q = c["requests"], c["q_heads"], c["kv_heads"], c["head_dim"], s["max_q"]
    table = s["table"].long().clamp(min=0)
    S = table.shape[1] * c["page"]
    kv = _values(s["cache"].codes[table], s["cache"].meta[table])  # [B, W, 2, H, page, D]
    k, v = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, B, H, S, D)
    lens, queries = s["kv"].long(), s["cu"].long().diff()
    i, t = torch.arange(Q, device="cuda")[None, :], torch.arange(S, device="cuda")
    row = (s["cu"][:-1].long()[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(B, Q, H, Hq // H, D).permute(0, 2, 3, 1, 4).reshape(B, H, -1, D)
    scores = (q @ k.transpose(-1, -2) * s["scale"]).view(B, H, Hq // H, Q, S)
    at = lens[:, None] - queries[:, None] + i
    seen = (t[None, None, :] <= at[..., None]) & (t[None, None, :] < lens[:, None, None])
    scores = scores.masked_fill(~seen[:, None, None], -torch.inf)
    p = torch.exp(scores - scores.amax(-1, keepdim=True).clamp(min=-3e38))
    total = p.sum(-1, keepdim=True)
    p = (p / torch.where(total > 0, total, 1)).view(B, H, -1, S)
    o = (p @ v).view(B, H, Hq // H, Q, D).permute(0, 3, 1, 2, 4).reshape(B, Q, Hq, D).half()
    b = torch.searchsorted(s["cu"][1:].contiguous(), torch.arange(s["q"].shape[0], device="cuda", dtype=torch.int32),
                           right=True)
    return {"out": o[b, torch.arange(s["q"].shape[0], device="cuda") - s["cu"].long()[b]]}


_plain = {"assign": _plain_assign, "append": _plain_append, "norm": _plain_norm, "attend": _plain_attend}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    if case["op"] == "assign":  # whole numbers only
        return None
    s = prepare(case, seed)
    return {"append": _exact_append, "norm": _exact_norm, "attend": _exact_attend}[case["op"]](s)


def _exact_append(s):
    c, R, D = s["case"], s["case"]["rotary"], s["case"]["head_dim"]
    x = s["qkv"].double()
    angles = s["rope"].double()[s["pos"].long()]
    turn = torch.complex(angles[:, :R // 2], angles[:, R // 2:])[:, None]
    heads = c["q_heads"] + c["kv_heads"]
    z = torch.complex(x[:, :heads, :R // 2], x[:, :heads, R // 2:R]) * turn
    x[:, :heads, :R] = torch.cat((z.real, z.imag), -1)
    q, rows = x[:, :c["q_heads"]].clone(), x[:, c["q_heads"]:].half().double()
    lo, hi = rows.min(-1).values.minimum(torch.zeros(())), rows.max(-1).values.maximum(torch.zeros(()))
    step = ((hi - lo) / 15).half().double()[..., None]
    zero = torch.nan_to_num(torch.round(-lo[..., None] / step)).clamp(0, 15)
    value = torch.nan_to_num((torch.round(rows / step) + zero).clamp(0, 15) - zero) * step
    k, v = value.clamp(-HALF_MAX, HALF_MAX).split(c["kv_heads"], 1)
    return {"q": q, "k": k, "v": v}


def _exact_norm(s):
    def unit(a):
        return a / (a.pow(2).sum(-1, keepdim=True) / a.shape[-1] + s["eps"]).sqrt()

    u = s["x"].double()
    u = unit(u) * s["w_post"].double() if s["w_post"] is not None else u
    u = u * s["gate"].double() if s["gate"] is not None else u
    r = s["r"].double() + s["scale"] * u
    y = unit(r.to(s["r"].dtype).double()) * s["w"].double()
    if s["case"]["quantize"]:
        y = y.half().double().unflatten(-1, (-1, 128))
        step = y.abs().max(-1, keepdim=True).values.div(127).float().double()
        y = (torch.nan_to_num(torch.round(y / step)).clamp(-127, 127) * step).flatten(-2)
    return {"r": r, "y": y}


def _exact_attend(s):
    c = s["case"]
    H, D, group = c["kv_heads"], c["head_dim"], c["q_heads"] // c["kv_heads"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, (n, m) in enumerate(zip(*_lengths(c))):
        pages = s["table"][b, :-(-n // c["page"])].long()
        first = int(s["cu"][b])
        for h in range(H):
            codes = s["cache"].codes[pages, :, h].transpose(0, 1).reshape(2, -1, D // 2)[:, :n]
            meta = s["cache"].meta[pages, :, h].transpose(0, 1).reshape(2, -1)[:, :n]
            value = torch.empty((2, n, D), dtype=torch.float64, device="cuda")
            value[..., 0::2], value[..., 1::2] = codes.bitwise_and(15), codes.div(16, rounding_mode="floor")
            value -= meta.div(65536, rounding_mode="floor")[..., None]
            value *= meta.remainder(65536).to(torch.int16).view(torch.float16).double()[..., None]
            q = s["q"][first:first + m, h * group:(h + 1) * group].double()
            a = torch.einsum("ihd,td->iht", q, value[0]) * s["scale"]
            late = torch.arange(n, device="cuda")[None, :] > n - m + torch.arange(m, device="cuda")[:, None]
            a.masked_fill_(late[:, None], -math.inf)
            out[first:first + m, h * group:(h + 1) * group] = torch.einsum("iht,td->ihd", a.softmax(-1), value[1])
    return {"out": out}
