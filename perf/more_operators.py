"""The measured cases of the 8-bit operators: linears in 8-bit integers with a
scale per token and channel, norms of query and key heads with their rotation,
and the paged 8-bit KV cache (append, read-back, attention).  `run` computes each
in plain torch, or with `own` through the package's entry points."""
import math

import torch

own = False

HALF_MAX = 65504.0
BLOCK = 16  # tokens of one scale


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one token through Llama-3.1-8B's qkv: latency and the weights' bytes
        {"name": "linear_decode_1", "op": "linear", "tokens": 1, "inner": 4096, "channels": 6144, "bias": False},
        # a decode batch of odd size through the 8B gate_up
        {"name": "linear_batch_37", "op": "linear", "tokens": 37, "inner": 4096, "channels": 28672, "bias": False},
        # a prompt through q_proj, with the bias of the projections that have one
        {"name": "linear_prompt_512", "op": "linear", "tokens": 512, "inner": 4096, "channels": 4096, "bias": True},
        # a long prompt, an odd number of tokens, through the 8B down projection
        {"name": "linear_prompt_2047", "op": "linear", "tokens": 2047, "inner": 14336, "channels": 4096,
         "bias": False},
        # a decode step's query and key heads
        {"name": "head_norm_decode_16", "op": "head_norm", "tokens": 16, "q_heads": 32, "kv_heads": 8,
         "head_dim": 128, "rotary": 128},
        # a chunk of prompts at Llama-3.1-70B's heads, half of the channels rotated
        {"name": "head_norm_prompt_4099", "op": "head_norm", "tokens": 4099, "q_heads": 64, "kv_heads": 8,
         "head_dim": 128, "rotary": 64},
        # one token of each of 32 requests, with the heads' norms, into blocks that hold older tokens
        {"name": "append_decode_32", "op": "append", "requests": 32, "new": 1, "q_heads": 32, "kv_heads": 8,
         "head_dim": 128, "rotary": 128, "page": 64, "norm": True},
        # chunks of prompts that begin and end within blocks
        {"name": "append_prompt_1367", "op": "append", "requests": 3, "new": 1367, "q_heads": 64, "kv_heads": 8,
         "head_dim": 128, "rotary": 128, "page": 16, "norm": False},
        # one request's decode step at a short context: latency
        {"name": "attend_decode_1", "op": "attend", "requests": 1, "query": 1, "short": 1003, "long": 1003,
         "q_heads": 32, "kv_heads": 8, "head_dim": 128, "page": 16},
        # a batch of requests of very different lengths, one token each
        {"name": "attend_decode_64", "op": "attend", "requests": 64, "query": 1, "short": 100, "long": 8100,
         "q_heads": 32, "kv_heads": 8, "head_dim": 128, "page": 64},
        # few requests with very long contexts at Llama-3.1-70B's heads
        {"name": "attend_decode_long", "op": "attend", "requests": 4, "query": 1, "short": 100000, "long": 131071,
         "q_heads": 64, "kv_heads": 8, "head_dim": 128, "page": 128},
        # chunks of prompts behind cached prefixes
        {"name": "attend_prompt_1024", "op": "attend", "requests": 2, "query": 1024, "short": 5000, "long": 8192,
         "q_heads": 32, "kv_heads": 8, "head_dim": 128, "page": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "head_norm", "append", "attend", "attend", "attend"])
    page = rng.choice([16, 32, 64, 128])
    heads = rng.choice([(32, 8, 128), (64, 8, 128), (16, 16, 64), (8, 1, 128), (40, 8, 128), (16, 2, 64)])
    shape = {"q_heads": heads[0], "kv_heads": heads[1], "head_dim": heads[2]}
    if op == "linear":
        inner = 16 * _log(rng, 16, 896)
        channels = _log(rng, 200, 28672)
        most = 2047 * 14336 * 4096 // (inner * channels)
        return {"op": op, "tokens": _log(rng, 1, min(4096, most)), "inner": inner, "channels": channels,
                "bias": rng.random() < 0.5}
    if op == "head_norm":
        return {"op": op, "tokens": _log(rng, 1, 4096), **shape, "rotary": rng.choice([heads[2], heads[2] // 2])}
    if op == "append":
        new = rng.choice([1, 1, _log(rng, 2, 2048)])
        return {"op": op, "requests": _log(rng, 1, max(2, 4096 // new // 2)), "new": new, **shape,
                "rotary": rng.choice([heads[2], heads[2] // 2]), "page": page, "norm": rng.random() < 0.5}
    if rng.random() < 0.7:  # decode and checks of a few proposed tokens
        requests = _log(rng, 1, 128)
        query = rng.choice([1, 1, 2, 3, 5])
        long = max(query, _log(rng, 16, min(131072, 430000 // requests)))
    else:  # chunks of prompts
        requests = rng.choice([1, 1, 2, 3, 4])
        query = _log(rng, 8, 36864 // heads[0] // requests)
        long = query + _log(rng, 1, 8192)
    return {"op": op, "requests": requests, "query": query, "short": max(query, long // rng.choice([1, 2, 7])),
            "long": long, **shape, "page": page}


def _spread(n, lo, hi):
    """n whole numbers in [lo, hi], unevenly spread, the first one hi."""
    return [hi - int((hi - lo) * (i * 0.6180339887498949 % 1.0)) for i in range(n)]


def _lengths(case):
    """Cached tokens of each request (its new ones among them) and its queries."""
    kv = _spread(case["requests"], case["short"], case["long"])
    if case["query"] <= 8:
        return kv, [case["query"]] * case["requests"]
    return kv, [min(k, q) for k, q in zip(kv, _spread(case["requests"], case["query"] * 3 // 4, case["query"]))]


def _appended(case):
    """(tokens before, new tokens) of each request's first touched block and what follows."""
    return [((7 * i + 5) % BLOCK, case["new"]) for i in range(case["requests"])]


def work(case):
    if case["op"] == "linear":
        M, K, N = case["tokens"], case["inner"], case["channels"]
        return {"bytes": N * K + 4 * N + 2 * M * K + 2 * M * N + (2 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    D = case["head_dim"]
    q, kv = case["q_heads"] * D, case["kv_heads"] * D
    if case["op"] == "head_norm":
        return {"bytes": case["tokens"] * (4 * (q + kv) + 4 * case["rotary"] + 4) + 4 * D,
                "flops": case["tokens"] * 8 * (q + kv)}
    if case["op"] == "append":
        T = case["requests"] * case["new"]
        back = sum(old + new for old, new in _appended(case))  # read back: older tokens of the blocks, too
        blocks = sum(-(-(old + new) // BLOCK) for old, new in _appended(case))
        per = 4 * q + 4 * kv + 4 * case["rotary"] + 12 + 2 * kv  # heads in, queries and codes out
        return {"bytes": T * per + back * (6 * kv + 8) + blocks * 2 * 2 * 4 * case["kv_heads"],
                "flops": T * (8 * (q + kv) + 6 * kv)}
    kv, qs = _lengths(case)
    H = case["q_heads"]
    pairs = sum(q * (k - q) + q * (q + 1) // 2 for k, q in zip(kv, qs))
    cache = sum(kv) * 2 * case["kv_heads"] * D + sum(-(-k // BLOCK) for k in kv) * 2 * case["kv_heads"] * 4
    return {"bytes": cache + 4 * sum(qs) * H * D + 4 * sum(-(-k // case["page"]) for k in kv),
            "flops": 4 * pairs * D * H}


# ------------------------------------------------------------------ inputs

def _rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _table(far, R):
    angle = torch.outer(torch.arange(far, dtype=torch.float64, device="cuda"),
                        500000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R))
    return torch.cat((angle.cos(), angle.sin()), 1).to(torch.float32)


class _Cache:
    """The parts of an 8-bit paged cache: codes uint8 [pages, 2, heads, page,
    dim] (128 is zero) and scales fp32 [pages, 2, heads, page / 16]."""

    def __init__(self, codes, scales):
        self.codes, self.scales = codes, scales


def _cache(g, pages, heads, page, dim):
    shape = (pages, 2, heads, page, dim)
    codes = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8) >> 1
    # the sum of two uniform numbers: spread like the codes of normal values
    codes += torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8) >> 1
    scales = 0.01 + 0.02 * torch.rand(shape[:3] + (page // BLOCK,), generator=g, device="cuda")
    return _Cache(codes + 1, scales)


def _handle(cache):
    from mixed_precision_quantized_act_b200 import KV8Cache
    return KV8Cache(cache.codes, cache.scales)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "linear":
        M, K, N = case["tokens"], case["inner"], case["channels"]
        outlier = 1 + 19 * (torch.rand(K, generator=g, device="cuda") < 0.01)
        s["x"] = (_rand(g, M, K) * outlier).to(torch.float16)
        s["codes"] = (_rand(g, N, K) * 32).round().clamp(-127, 127).to(torch.int8)
        s["s_w"] = 0.0004 + 0.0008 * torch.rand(N, generator=g, device="cuda")
        s["bias"] = _rand(g, N).to(torch.float16) if case["bias"] else None
        s["y"] = torch.empty((M, N), dtype=torch.float16, device="cuda")
        return s
    p, D, Hq, H = case.get("page", 0), case["head_dim"], case["q_heads"], case["kv_heads"]
    if case["op"] == "attend":
        kv, qs = _lengths(case)
        used = [-(-k // p) for k in kv]
        W, pages = max(used), sum(used) + 3
        s["cache"] = _cache(g, pages, H, p, D)
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        ends = _ints(used).cumsum(0)
        j = torch.arange(W, device="cuda")[None, :]
        first = (ends - _ints(used))[:, None]
        s["table"] = torch.where(j < _ints(used)[:, None], order[(first + j).clamp(max=pages - 1)], -1)
        s["kv"], s["cu"] = _ints(kv), _ints([sum(qs[:i]) for i in range(len(qs) + 1)])
        s["max_q"] = max(qs)
        s["q"] = _rand(g, sum(qs), Hq, D).to(torch.float16)
        s["out"] = torch.empty_like(s["q"])
        s["scale"] = 1.0 / math.sqrt(D)
        return s
    T = case["tokens"] if case["op"] == "head_norm" else case["requests"] * case["new"]
    outlier = 1 + 7 * (torch.rand(D, generator=g, device="cuda") < 0.03)  # a few large channels, as in real keys
    s["qkv"] = (_rand(g, T, Hq + 2 * H, D) * outlier).to(torch.float16)
    s["w_q"], s["w_k"] = ((1 + 0.2 * _rand(g, D)).to(torch.float16) for _ in range(2))
    s["eps"] = 1e-6
    s["rope"] = _table(16384, case["rotary"])
    s["pos"] = torch.randint(0, 16384, (T,), generator=g, device="cuda", dtype=torch.int32)
    s["q_out"] = torch.empty((T, Hq, D), dtype=torch.float16, device="cuda")
    if case["op"] == "head_norm":
        s["k_out"] = torch.empty((T, H, D), dtype=torch.float16, device="cuda")
        return s
    # each request's touched blocks stand one behind the other in pages of its own, older tokens at their front
    each = [-(-(old + new) // p) for old, new in _appended(case)]
    order = torch.randperm(sum(each) + 2, generator=g, device="cuda")
    s["cache"] = _cache(g, sum(each) + 2, H, p, D)
    new_slots, back, at = [], [], 0
    for (old, new), n in zip(_appended(case), each):
        row = torch.arange(old + new, device="cuda")
        slot = order[at + row // p] * p + row % p
        new_slots.append(slot[old:])
        back.append(slot)
        at += n
    s["slots"], s["back"] = torch.cat(new_slots), torch.cat(back)
    s["k_out"], s["v_out"] = (torch.empty((s["back"].numel(), H, D), dtype=torch.float16, device="cuda")
                              for _ in range(2))
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _own_linear(s):
    import mixed_precision_quantized_act_b200 as mx
    if "weights" not in s:
        s["weights"] = mx.W8Weights(s["codes"], s["s_w"])
        s["workspace"] = mx.w8a8_linear_workspace(s["x"].shape[0], s["weights"])
    mx.w8a8_linear_into(s["x"], s["weights"], s["y"], s["workspace"], bias=s["bias"])
    return {"y": s["y"]}


def _own_head_norm(s):
    import mixed_precision_quantized_act_b200 as mx
    c = s["case"]
    q, k, _ = s["qkv"].split((c["q_heads"], c["kv_heads"], c["kv_heads"]), 1)
    mx.head_norm_rope_into(q, s["q_out"], s["w_q"], k=k, k_out=s["k_out"], w_k=s["w_k"], positions=s["pos"],
                           rope=s["rope"], eps=s["eps"])
    return {"q": s["q_out"], "k": s["k_out"]}


def _own_append(s):
    import mixed_precision_quantized_act_b200 as mx
    if "handle" not in s:
        s["handle"] = _handle(s["cache"])
    c = s["case"]
    q, k, v = s["qkv"].split((c["q_heads"], c["kv_heads"], c["kv_heads"]), 1)
    norm = {"w_q": s["w_q"], "w_k": s["w_k"], "eps": s["eps"]} if c["norm"] else {}
    mx.kv8_append_into(k, v, s["slots"], s["handle"], q=q, q_out=s["q_out"], positions=s["pos"], rope=s["rope"], **norm)
    mx.kv8_read_into(s["back"], s["handle"], s["k_out"], s["v_out"])
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def _own_attend(s):
    import mixed_precision_quantized_act_b200 as mx
    if "handle" not in s:
        s["handle"] = _handle(s["cache"])
        s["workspace"] = mx.kv8_attention_workspace(s["case"]["requests"], s["max_q"], s["case"]["q_heads"],
                                                    s["handle"], s["table"].shape[1])
    mx.kv8_attention_into(s["q"], s["handle"], s["table"], s["kv"], s["cu"], s["max_q"], s["out"], s["workspace"],
                          scale=s["scale"])
    return {"out": s["out"]}


_own = {"linear": _own_linear, "head_norm": _own_head_norm, "append": _own_append, "attend": _own_attend}


def _steps(amax):
    return amax / torch.full_like(amax, 127.0)


def _plain_linear(s):
    x = s["x"].float()
    step = _steps(x.abs().amax(-1, keepdim=True))
    a = (x / torch.where(step > 0, step, 1)).round().clamp(-127, 127)
    y = (a @ s["codes"].float().t()) * step * s["s_w"]
    return {"y": (y if s["bias"] is None else y + s["bias"].float()).half()}


def _turned(x, w, eps, rope, R):
    """Each head normalized (w not None) and its first R channels rotated by halves: fp32, one rounding to fp16."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.float()
    cos, sin = rope[:, None, :R // 2], rope[:, None, R // 2:]
    a, b = x[..., :R // 2], x[..., R // 2:R]
    return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., R:]), -1).half()


def _plain_head_norm(s):
    c = s["case"]
    q, k, _ = s["qkv"].split((c["q_heads"], c["kv_heads"], c["kv_heads"]), 1)
    rope = s["rope"][s["pos"].long()]
    return {"q": _turned(q, s["w_q"], s["eps"], rope, c["rotary"]),
            "k": _turned(k, s["w_k"], s["eps"], rope, c["rotary"])}


def _kept(cache, slots, page):
    """fp32 keys and values [slots, 2, heads, dim] of the cached rows."""
    at, row = slots // page, slots % page
    return (cache.codes[at, :, :, row].float() - 128) * cache.scales[at, :, :, row // BLOCK][..., None]


def _plain_append(s):
    c, cache = s["case"], s["cache"]
    q, k, v = s["qkv"].split((c["q_heads"], c["kv_heads"], c["kv_heads"]), 1)
    rope = s["rope"][s["pos"].long()]
    w_q, w_k = (s["w_q"], s["w_k"]) if c["norm"] else (None, None)
    kv = torch.stack((_turned(k, w_k, s["eps"], rope, c["rotary"]), v), 1).float()
    blocks, mine = torch.unique(s["slots"] // BLOCK, return_inverse=True)
    per = c["page"] // BLOCK
    page, sub = blocks // per, blocks % per
    amax = torch.zeros((blocks.numel(),) + kv.shape[1:3], device="cuda")
    amax.index_reduce_(0, mine, kv.abs().amax(-1), "amax")
    anew = torch.zeros(blocks.numel(), device="cuda").index_fill_(0, mine[s["slots"] % BLOCK == 0], 1)[:, None, None] > 0
    before = torch.where(anew, 0, cache.scales[page, :, :, sub])
    step = torch.maximum(before, _steps(amax))
    rows = sub[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")
    ratio = (before / torch.where(step > 0, step, 1))[:, None, :, :, None]
    old = cache.codes[page[:, None], :, :, rows]
    grown = (step > before)[:, None, :, :, None] & ~anew[:, None, :, :, None]
    cache.codes[page[:, None], :, :, rows] = torch.where(
        grown, ((old.float() - 128) * ratio).round().clamp(-127, 127) + 128, old.float()).to(torch.uint8)
    cache.scales[page, :, :, sub] = step
    mine_step = step[mine][..., None]
    code = (kv / torch.where(mine_step > 0, mine_step, 1)).round().clamp(-127, 127) + 128
    cache.codes[s["slots"] // c["page"], :, :, s["slots"] % c["page"]] = code.to(torch.uint8)
    kept = _kept(cache, s["back"], c["page"]).clamp(-HALF_MAX, HALF_MAX).half()
    return {"q": _turned(q, w_q, s["eps"], rope, c["rotary"]), "k": kept[:, 0], "v": kept[:, 1]}


def _plain_attend(s):
    c = s["case"]
    B, Hq, H, D, Q = c["requests"], c["q_heads"], c["kv_heads"], c["head_dim"], s["max_q"]
    table = s["table"].long().clamp(min=0)
    S = table.shape[1] * c["page"]
    kv = s["cache"].codes[table].float() - 128  # [B, W, 2, H, page, D]
    kv *= s["cache"].scales[table].repeat_interleave(BLOCK, -1)[..., None]
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


_plain = {"linear": _plain_linear, "head_norm": _plain_head_norm, "append": _plain_append, "attend": _plain_attend}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "head_norm": _exact_heads, "append": _exact_append, "attend": _exact_attend}[
        case["op"]](s)


def _codes64(x, step):
    """Nearest whole multiples of `step` (an fp32 number): the quotient is an fp32 one."""
    return torch.nan_to_num(torch.round((x / step).float().double()), nan=0.0).clamp(-127, 127)


def _exact_linear(s):
    x = s["x"].double()
    step = x.abs().max(-1, keepdim=True).values.div(127).float().double()
    y = torch.einsum("mk,nk->mn", _codes64(x, step), s["codes"].double())
    y = y * (step * s["s_w"].double())
    return {"y": y if s["bias"] is None else y + s["bias"].double()}


def _heads64(x, w, s):
    R = s["case"]["rotary"]
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]).sqrt() * w.double()
    angles = s["rope"].double()[s["pos"].long()]
    turn = torch.complex(angles[:, :R // 2], angles[:, R // 2:])[:, None]
    z = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * turn
    return torch.cat((z.real, z.imag, x[..., R:]), -1)


def _exact_heads(s):
    c = s["case"]
    q, k, _ = s["qkv"].split((c["q_heads"], c["kv_heads"], c["kv_heads"]), 1)
    return {"q": _heads64(q, s["w_q"], s), "k": _heads64(k, s["w_k"], s)}


def _exact_append(s):
    c, H, p = s["case"], s["case"]["kv_heads"], s["case"]["page"]
    q, k, v = s["qkv"].split((c["q_heads"], H, H), 1)
    norm = c["norm"]
    k = _heads64(k, s["w_k"] if norm else None, s).half().double()
    out = {"q": _heads64(q, s["w_q"] if norm else None, s)}
    cache = s["cache"]
    for kind, (name, x) in enumerate((("k", k), ("v", v.double()))):
        values, first, seen = [], 0, 0
        for old, new in _appended(c):
            slots = s["back"][seen:seen + old + new]
            at, row = slots // p, slots % p
            code = cache.codes[at, kind, :, row].double() - 128  # [rows, H, D]
            scale = cache.scales[at, kind, :, row // BLOCK].double()
            fresh = x[first:first + new]
            pad = -(old + new) % BLOCK
            amax = torch.cat((torch.zeros(old, H, device="cuda", dtype=torch.float64), fresh.abs().amax(-1),
                              torch.zeros(pad, H, device="cuda", dtype=torch.float64)))
            step = amax.view(-1, BLOCK, H).amax(1).div(127).float().double()
            if old:
                step[0] = torch.maximum(step[0], scale[0])
            step = step.repeat_interleave(BLOCK, 0)[:old + new, :, None]
            ratio = (scale[..., None] / step).float().double()
            code = (code * ratio).float().double().round().clamp(-127, 127)
            code[old:] = _codes64(fresh, step[old:])
            values.append((code * step).clamp(-HALF_MAX, HALF_MAX))
            first, seen = first + new, seen + old + new
        out[name] = torch.cat(values)
    return out


def _exact_attend(s):
    c = s["case"]
    H, D, group = c["kv_heads"], c["head_dim"], c["q_heads"] // c["kv_heads"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, (n, m) in enumerate(zip(*_lengths(c))):
        pages = s["table"][b, :-(-n // c["page"])].long()
        first = int(s["cu"][b])
        for h in range(H):
            codes = s["cache"].codes[pages, :, h].transpose(0, 1).reshape(2, -1, BLOCK, D)
            scales = s["cache"].scales[pages, :, h].transpose(0, 1).reshape(2, -1, 1, 1)
            value = (codes.double().sub(128) * scales.double()).flatten(1, 2)[:, :n]
            q = s["q"][first:first + m, h * group:(h + 1) * group].double()
            a = torch.einsum("ihd,td->iht", q, value[0]) * s["scale"]
            late = torch.arange(n, device="cuda")[None, :] > n - m + torch.arange(m, device="cuda")[:, None]
            a.masked_fill_(late[:, None], -math.inf)
            out[first:first + m, h * group:(h + 1) * group] = torch.einsum("iht,td->ihd", a.softmax(-1), value[1])
    return {"out": out}
