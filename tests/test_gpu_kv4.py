"""The paged 4-bit KV cache on the GPU: page assignment, append, read-back and
attention against plain restatements of their definitions.  GPU only."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mixed_precision_quantized_act_b200 as mx  # noqa: E402
from mixed_precision_quantized_act_b200 import _lib  # noqa: E402
from tests import kv4_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.load()
    return torch.device("cuda:0")


# ------------------------------------------------------------------ assignment

def _assign_ref(ctx, new, table, free, count, page, T):
    """Straight loops over requests and tokens."""
    B, W = table.shape
    status = 0
    add = []
    for c, n in zip(ctx, new):
        if c < 0 or n < 0:
            status |= 8
            continue
        add.append(-(-(c + n) // page) + -c // page)
        if -(-(c + n) // page) > W:
            status |= 2
    total = sum(n for c, n in zip(ctx, new) if c >= 0 and n >= 0)
    status |= (1 if sum(add) > count or count > len(free) else 0) | (4 if total > T else 0)
    slots, pos = np.full(T, -1, np.int64), np.full(T, -1, np.int32)
    if status:
        return list(ctx), [0] * (B + 1), slots, pos, table.copy(), count, status
    table, t, cu = table.copy(), 0, [0]
    for b in range(B):
        for j in range(-(-ctx[b] // page), -(-(ctx[b] + new[b]) // page)):
            count -= 1
            table[b, j] = free[count]
        for i in range(new[b]):
            pos[t] = ctx[b] + i
            slots[t] = int(table[b, pos[t] // page]) * page + pos[t] % page
            t += 1
        cu.append(t)
    return [c + n for c, n in zip(ctx, new)], cu, slots, pos, table, count, 0


def _assign(dev, ctx, new, table, free, count, page, T, in_place=False, stream=None):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    c, n, left = i32(list(ctx)), i32(list(new)), i32([count])
    t, f = torch.from_numpy(table).to(dev), i32(list(free))
    seq = c if in_place else torch.full_like(c, -7)
    out = left if in_place else torch.full_like(left, -7)
    cu = torch.full((len(ctx) + 1,), -7, dtype=torch.int32, device=dev)
    slots = torch.full((T,), -7, dtype=torch.int64, device=dev)
    pos = torch.full((T,), -7, dtype=torch.int32, device=dev)
    status = torch.full((1,), -7, dtype=torch.int32, device=dev)
    mx.kv4_assign_into(c, n, t, f, left, page, seq, cu, slots, pos, out, status)
    mx.sync_status()
    return (seq.tolist(), cu.tolist(), slots.cpu().numpy(), pos.cpu().numpy(), t.cpu().numpy(), int(out), int(status))


def _same(got, want):
    assert got[0] == list(want[0]) and got[1] == list(want[1])
    assert np.array_equal(got[2], want[2]) and np.array_equal(got[3], want[3])
    assert np.array_equal(got[4], want[4])
    assert got[5:] == tuple(want[5:])


@pytest.mark.parametrize("B,top,ctx_top,page,pad", [
    (1, 1, 0, 16, 0), (1, 1, 16, 16, 3), (3, 5, 40, 16, 0), (64, 1, 300, 64, 7), (100, 0, 50, 32, 5),
    (33, 400, 999, 128, 11), (1025, 3, 60, 16, 0), (5000, 2, 33, 256, 9), (16384, 1, 20, 16, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_assign_matches_loops(dev, B, top, ctx_top, page, pad, in_place):
    rng = np.random.default_rng(B + top)
    ctx = rng.integers(0, ctx_top + 1, B).tolist()
    new = rng.integers(0, top + 1, B).tolist()
    W = -(-(ctx_top + top) // page) + 1
    ids = rng.permutation(2 * B * W).astype(np.int32)
    table = ids[:B * W].reshape(B, W).copy()
    used = np.arange(W)[None, :] < -(-np.array(ctx)[:, None] // page)
    table[~used] = -3  # entries behind a request's pages hold anything
    free, T = ids[B * W:].tolist(), sum(new) + pad
    want = _assign_ref(ctx, new, table, free, len(free), page, T)
    assert want[-1] == 0
    _same(_assign(dev, ctx, new, table, free, len(free), page, T, in_place), want)


@pytest.mark.parametrize("ctx,new,W,count,T,status", [
    ([10, 20], [10, 1], 2, 0, 20, 1),        # one page lacking, none free
    ([10, 20], [10, 1], 2, 9, 20, 1),        # more pages said to be free than the stack has
    ([10, 31], [1, 2], 2, 3, 20, 2),         # a third page for a table of two
    ([10, 20], [10, 1], 2, 3, 10, 4),        # eleven tokens for ten slots
    ([10, -1], [1, 1], 2, 3, 20, 8),
    ([10, 20], [1, -5], 2, 3, 20, 8),
    ([0, 2 ** 31 - 1], [2 ** 31 - 1, 2 ** 31 - 1], 2, 3, 20, 1 + 2 + 4),
    ([10, 20], [0, 0], 2, 0, 0, 0)])
def test_assign_refuses_as_a_whole(dev, ctx, new, W, count, T, status):
    table = np.arange(2 * W, dtype=np.int32).reshape(2, W)
    want = _assign_ref(ctx, new, table, [50, 51, 52], count, 16, T)
    assert want[-1] == status
    _same(_assign(dev, ctx, new, table, [50, 51, 52], count, 16, T), want)


def test_assign_without_requests(dev):
    got = _assign(dev, [], [], np.zeros((0, 3), np.int32), [1, 2], 2, 16, 5)
    assert got[0] == [] and got[1] == [0] and (got[2] == -1).all() and got[5:] == (2, 0)


# ------------------------------------------------------------------ append and read

def _rand_kv(rng, T, heads, D):
    x = rng.standard_normal((T, heads, D)).astype(np.float32)
    x *= 1 + 7 * (rng.random(D) < 0.05)
    x[rng.random((T, heads)) < 0.05] = 0                 # zero rows
    x[rng.random((T, heads)) < 0.05] *= 1e-6             # scales near and below fp16's smallest
    return x.astype(np.float16)


@pytest.mark.parametrize("T", [1, 7, 130])
@pytest.mark.parametrize("Hq,H,D,rotary,page", [(8, 2, 128, 128, 64), (4, 4, 64, 64, 16), (3, 1, 128, 64, 128),
                                                (0, 3, 64, 16, 32), (5, 5, 64, 0, 256), (0, 1, 128, 0, 16)])
def test_append_bits_match_and_nothing_else_moves(dev, T, Hq, H, D, rotary, page):
    rng = np.random.default_rng(T * 1000 + D + rotary)
    pages = -(-T // page) + 2
    qkv = _rand_kv(rng, T, Hq + 2 * H + 1, D)            # one head more: rows are strided
    table = mx.rope_table(512, rotary, 500000.0, dev) if rotary else None
    pos = rng.integers(0, 512, T).astype(np.int32)
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    if T > 3:
        slots[T // 2] = -1                               # a token that is skipped
    cache = mx.kv4_cache(pages, H, D, page, dev)
    cache.codes.random_(0, 256)
    cache.meta.random_()
    codes0, meta0 = cache.codes.cpu().numpy(), cache.meta.cpu().numpy().view(np.uint32)
    x = torch.from_numpy(qkv).to(dev)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:Hq + 2 * H]
    q_out = torch.full((T, Hq, D), 9.0, dtype=torch.float16, device=dev) if Hq else None
    mx.kv4_append_into(k, v, torch.from_numpy(slots).to(dev), cache, q=q if Hq else None, q_out=q_out,
                       positions=torch.from_numpy(pos).to(dev) if rotary else None, rope=table)
    mx.sync_status()
    rot = qkv.copy()
    if rotary:
        rot[:, :Hq + H] = ref.rotate(qkv[:, :Hq + H], table.cpu().numpy(), pos, rotary)
    for kind, rows in ((0, rot[:, Hq:Hq + H]), (1, rot[:, Hq + H:Hq + 2 * H])):
        by, meta = ref.pack(*ref.quantize_row(rows))
        for t in range(T):
            if slots[t] >= 0:
                codes0[slots[t] // page, kind, :, slots[t] % page] = by[t]
                meta0[slots[t] // page, kind, :, slots[t] % page] = meta[t]
    assert np.array_equal(cache.codes.cpu().numpy(), codes0)
    assert np.array_equal(cache.meta.cpu().numpy().view(np.uint32), meta0)
    if Hq:
        want = rot[:, :Hq].copy()
        want[slots < 0] = 9.0
        assert np.array_equal(q_out.cpu().numpy().view(np.uint16), want.view(np.uint16))
    # read back: s (code - z), rounded once
    k_out = torch.full((T, H, D), 5.0, dtype=torch.float16, device=dev)
    v_out = torch.full_like(k_out, 5.0)
    mx.kv4_read_into(torch.from_numpy(slots).to(dev), cache, k_out, v_out)
    mx.sync_status()
    val = ref.values(torch.from_numpy(codes0), torch.from_numpy(meta0.view(np.int32))).clamp(-65504, 65504).half()
    for t in range(T):
        for kind, got in ((0, k_out), (1, v_out)):
            want = val[slots[t] // page, kind, :, slots[t] % page] if slots[t] >= 0 else torch.full((H, D), 5.0).half()
            assert torch.equal(got[t].cpu(), want)


def test_append_in_place_rotation_and_extremes(dev):
    rng = np.random.default_rng(3)
    T, H, D = 6, 2, 128
    x = _rand_kv(rng, T, 3 * H, D)
    x[0, H, 5], x[1, H, 9], x[2, 2 * H, 0] = np.nan, np.inf, -np.inf
    x[3, 2 * H, :] = 65504
    x[3, 2 * H, 1::2] = -65504
    x[4, 2 * H, :] = 6e-8                                # the smallest fp16 number: its scale rounds to 0
    q, k, v = (torch.from_numpy(x[:, i * H:(i + 1) * H].copy()).to(dev) for i in range(3))
    cache = mx.kv4_cache(2, H, D, 16, dev)
    slots = torch.arange(T, device=dev)
    table = mx.rope_table(64, D, device=dev)
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    mx.kv4_append_into(k, v, slots, cache, q=q, q_out=q, positions=pos, rope=table)
    mx.sync_status()
    rot = ref.rotate(x[:, :2 * H], table.cpu().numpy(), pos.cpu().numpy(), D)
    assert np.array_equal(q.cpu().numpy().view(np.uint16), rot[:, :H].view(np.uint16))
    kc, vc = (ref.quantize_row(r) for r in (rot[:, H:], x[:, 2 * H:]))
    meta = cache.meta.cpu().numpy().view(np.uint32)
    for kind, (c, s, z) in ((0, kc), (1, vc)):
        by, m = ref.pack(c, s, z)
        bad = np.isnan(s)
        got = meta[0, kind, :, :T].T
        assert np.array_equal(got[~bad], m[~bad])
        assert np.isnan(got[bad].astype(np.uint16).view(np.float16)).all() and (got[bad] >> 16 == 0).all()
        assert np.array_equal(cache.codes[0, kind, :, :T].permute(1, 0, 2).cpu().numpy(), by)
    k_out, v_out = torch.zeros_like(k), torch.zeros_like(v)
    mx.kv4_read_into(slots, cache, k_out, v_out)
    assert k_out[0, 0].isnan().all() and k_out[1, 0].isnan().all() and v_out[2, 0].isnan().all()
    # s = fp16(131008 / 15) = 8736, z = rne(7.498) = 7, codes 0 (rne(-7.498) + 7) and 14 (rne(7.498) + 7): +-7 steps
    assert bool(v_out[3].isfinite().all()) and float(v_out[3, 0].abs().max()) == 7 * 8736
    assert bool(k_out[0, 1].isfinite().all())


def test_read_stays_within_the_finite_values(dev):
    # all 65504: s = fp16(65504 / 15 = 4366.9) = 4368, z = 0, code 15; 15 * 4368 = 65520 would round to infinity
    x = torch.full((1, 1, 64), 65504.0, dtype=torch.float16, device=dev)
    cache, slots = mx.kv4_cache(1, 1, 64, 16, dev), torch.zeros(1, dtype=torch.int64, device=dev)
    mx.kv4_append_into(x, -x, slots, cache)
    k, v = torch.zeros_like(x), torch.zeros_like(x)
    mx.kv4_read_into(slots, cache, k, v)
    mx.sync_status()
    assert torch.equal(k, x) and torch.equal(v, -x)


@pytest.mark.parametrize("slot,pos", [(32, 0), (2 ** 40, 0), (3, 64), (3, -1)])
def test_append_skips_and_reports_what_is_out_of_range(dev, slot, pos):
    cache = mx.kv4_cache(2, 1, 64, 16, dev)
    kv = torch.ones((2, 1, 64), dtype=torch.float16, device=dev)
    slots = torch.tensor([1, slot], device=dev)
    mx.kv4_append_into(kv, kv, slots, cache, positions=torch.tensor([0, pos], dtype=torch.int32, device=dev),
                       rope=mx.rope_table(64, 64, device=dev))
    with pytest.raises(_lib.MixLLMError) as e:
        mx.sync_status()
    assert e.value.status == _lib.ERR_BOUNDS
    meta = cache.meta.clone()
    assert meta[0, 0, 0, 1] != 0
    meta[0, :, 0, 1] = 0
    assert not meta.any()
    if slot >= 32:
        out = torch.full((2, 1, 64), 7.0, dtype=torch.float16, device=dev)
        mx.kv4_read_into(slots, cache, out, out.clone())
        with pytest.raises(_lib.MixLLMError):
            mx.sync_status()
        assert (out[1] == 7).all()


# ------------------------------------------------------------------ attention

def _case(dev, kv, qs, Hq, H, D, page, seed=0, tail=0, wide=False, extra_width=1):
    """A cache of random codes whose unused rows and table entries hold
    garbage (NaN scales, pages that do not exist)."""
    g = torch.Generator().manual_seed(seed)
    used = [-(-n // page) for n in kv]
    pages, W = sum(used) + 2, max(used, default=0) + extra_width
    codes = torch.randint(0, 256, (pages, 2, H, page, D // 2), generator=g, dtype=torch.uint8)
    s = torch.rand((pages, 2, H, page), generator=g) * 0.3 + 0.05
    if wide:  # value scales over many orders of magnitude, some zero
        s[:, 1] = torch.exp2(torch.rand((pages, H, page), generator=g) * 30 - 24)
        s[:, 1][torch.rand((pages, H, page), generator=g) < 0.2] = 0
    z = torch.randint(0, 16, (pages, 2, H, page), generator=g, dtype=torch.int32)
    meta = (s.half().view(torch.int16).to(torch.int32) & 0xFFFF) | z << 16
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(kv), W), 2 ** 31 - 1, dtype=torch.int32)
    at = 0
    nan = torch.tensor(0x0FFF7E00, dtype=torch.int32)
    free = torch.ones((pages, page), dtype=torch.bool)
    for b, n in enumerate(kv):
        table[b, :used[b]] = order[at:at + used[b]]
        for j in range(used[b]):
            free[order[at + j], :n - j * page] = False
        at += used[b]
    meta = torch.where(free[:, None, None, :], nan, meta)
    cu = [0]
    for m in qs:
        cu.append(cu[-1] + m)
    q = torch.randn((cu[-1] + tail, Hq, D), generator=g).half()
    cache = mx.KV4Cache(codes.to(dev), meta.to(dev))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    return q, cache, table, i32(list(kv)), i32(cu)


def _check(dev, kv, qs, Hq, H, D, page, causal=True, scale=None, seed=0, tail=0, wide=False, max_q=None):
    q, cache, table, lens, cu = _case(dev, kv, qs, Hq, H, D, page, seed, tail, wide)
    scale = D ** -0.5 if scale is None else scale
    T = q.shape[0]
    out = torch.full((T, Hq, D), 77.0, dtype=torch.float16, device=dev)
    lse = torch.full((T, Hq), 77.0, dtype=torch.float32, device=dev)
    max_q = max(qs) if max_q is None else max_q
    ws = mx.kv4_attention_workspace(len(kv), max_q, Hq, cache, table.shape[1])
    args = (q.to(dev), cache, table.to(dev), lens, cu, max_q)
    mx.kv4_attention_into(*args, out, ws, scale, causal, lse)
    mx.sync_status()
    want, want_lse, tol = ref.attention(q, cache.codes.cpu(), cache.meta.cpu(), table, kv, cu.tolist(), scale, causal)
    n = int(cu[-1])
    got = out.cpu().double()
    off = (got[:n] - want[:n]).abs()
    assert (off <= tol[:n]).all(), (float((off / tol[:n].clamp(min=1e-30)).max()), float(off.max()))
    assert (got[n:] == 77).all() and (lse[n:] == 77).all()
    seen = want_lse[:n] > -float("inf")
    assert (lse[:n].cpu()[~seen] == -float("inf")).all()
    # lse: the relative errors of the probabilities' sum, and the rounding of the result
    far = (lse[:n].cpu().double() - want_lse[:n]).abs()[seen]
    assert (far <= 2.0 ** -18 * (1 + want_lse[:n].abs()[seen]) + 64 * D * 2.0 ** -24).all()
    # the workspace is ready again, and the result does not depend on timing
    again = torch.full_like(out, 77.0)
    mx.kv4_attention_into(*args, again, ws, scale, causal)
    mx.sync_status()
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))
    assert not ws[:4096].any()


@pytest.mark.parametrize("kv", [[1], [0], [2, 15, 16, 17], [127, 128, 129, 130], [0, 300, 1, 0, 257], [4097, 1, 700]],
                         ids=str)
@pytest.mark.parametrize("Hq,H,D,page", [(8, 2, 128, 64), (4, 4, 64, 16), (8, 1, 128, 128), (6, 2, 64, 256),
                                         (2, 1, 128, 32)])
def test_attention_of_single_tokens(dev, kv, Hq, H, D, page):
    _check(dev, kv, [1] * len(kv), Hq, H, D, page, seed=len(kv))


@pytest.mark.parametrize("kv,qs", [([3, 0, 40, 129], [3, 0, 2, 5]), ([2, 1], [5, 1]), ([200, 17], [8, 8]),
                                   ([1000], [2]), ([0, 0], [3, 1])], ids=str)
@pytest.mark.parametrize("Hq,H,D,page", [(4, 2, 128, 16), (10, 1, 64, 64), (20, 1, 128, 64), (3, 3, 64, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_of_few_tokens(dev, kv, qs, Hq, H, D, page, causal):
    _check(dev, kv, qs, Hq, H, D, page, causal, seed=sum(kv), tail=3)


@pytest.mark.parametrize("kv,qs", [([70], [70]), ([300, 131], [150, 131]), ([515], [33]), ([90, 5, 64], [90, 9, 1])],
                         ids=str)
@pytest.mark.parametrize("Hq,H,D,page", [(4, 1, 128, 64), (2, 2, 64, 16), (3, 1, 128, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_of_prompts(dev, kv, qs, Hq, H, D, page, causal):
    _check(dev, kv, qs, Hq, H, D, page, causal, seed=sum(qs), tail=1)


def test_attention_over_a_long_context(dev):
    _check(dev, [20011], [1], 4, 2, 128, 64, seed=5)
    _check(dev, [9000, 30, 12345], [1, 1, 1], 2, 1, 64, 16, seed=6)


def test_attention_with_more_requests_than_threads(dev):
    rng = np.random.default_rng(1)
    kv = rng.integers(0, 60, 700).tolist()
    _check(dev, kv, [1] * 700, 2, 1, 64, 16, seed=7)


@pytest.mark.parametrize("D", [64, 128])
def test_attention_with_value_scales_of_all_sizes(dev, D):
    _check(dev, [400, 129], [1, 2], 4, 2, D, 64, seed=8, wide=True)


@pytest.mark.parametrize("scale", [1e-4, 3.0, -0.5])
def test_attention_with_other_scales(dev, scale):
    _check(dev, [333], [1], 4, 1, 128, 64, scale=scale, seed=9)


def test_attention_takes_strided_tensors(dev):
    kv, qs, Hq, H, D, page = [150, 60], [2, 1], 4, 2, 128, 64
    q, cache, table, lens, cu = _case(dev, kv, qs, Hq, H, D, page)
    wide = torch.zeros((3, Hq + 2, D), dtype=torch.float16, device=dev)
    wide[:, 1:1 + Hq] = q.to(dev)
    out = torch.full((3, Hq + 3, D), 77.0, dtype=torch.float16, device=dev)
    big = torch.full((2, table.shape[1] + 5), -1, dtype=torch.int32, device=dev)
    big[:, :table.shape[1]] = table.to(dev)
    ws = mx.kv4_attention_workspace(2, 2, Hq, cache, table.shape[1])
    mx.kv4_attention_into(wide[:, 1:1 + Hq], cache, big[:, :table.shape[1]], lens, cu, 2, out[:, 2:2 + Hq], ws)
    want = mx.kv4_attention(q.to(dev), cache, table.to(dev), lens, cu, 2)
    mx.sync_status()
    assert torch.equal(out[:, 2:2 + Hq], want)
    assert (out[:, :2] == 77).all() and (out[:, 2 + Hq:] == 77).all()


def test_attention_nan_rows_poison_only_who_sees_them(dev):
    kv, qs, Hq, H, D, page = [200], [3], 4, 2, 128, 64
    q, cache, table, lens, cu = _case(dev, kv, qs, Hq, H, D, page)
    t = 198  # seen by the second and third query, not by the first
    for kind in (0, 1):
        meta = cache.meta.clone()
        meta[table[0, t // page], kind, 1, t % page] = 0x7FFF
        out = mx.kv4_attention(q.to(dev), mx.KV4Cache(cache.codes, meta), table.to(dev), lens, cu, 3)
        mx.sync_status()
        assert out[0].isfinite().all()
        assert out[1:, 2:].isnan().all() and out[1:, :2].isfinite().all()


def test_attention_reports_pages_and_lengths_out_of_range(dev):
    kv, qs, Hq, H, D, page = [300, 100], [1, 2], 4, 2, 128, 64
    q, cache, table, lens, cu = _case(dev, kv, qs, Hq, H, D, page)

    def run(table, lens, cu, max_q=2):
        out = torch.full(q.shape, 77.0, dtype=torch.float16, device=dev)
        ws = mx.kv4_attention_workspace(2, max_q, Hq, cache, table.shape[1])
        mx.kv4_attention_into(q.to(dev), cache, table.to(dev), lens, cu, max_q, out, ws)
        with pytest.raises(_lib.MixLLMError) as e:
            mx.sync_status()
        assert e.value.status == _lib.ERR_BOUNDS
        assert not ws[:4096].any()
        return out.cpu().double()

    for wrong in (-1, cache.pages, 2 ** 31 - 1, -2 ** 31):  # the tokens of a bad page are not seen
        bad = table.clone()
        bad[0, 2] = wrong
        out = run(bad, lens, cu)
        want, _, tol = ref.attention(q, cache.codes.cpu(), cache.meta.cpu(), bad, kv, cu.tolist(), D ** -0.5, True)
        assert ((out - want).abs() <= tol).all()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    # A request with such lengths gets nothing; the others get theirs.  (Compared with the reference and not
    # bit by bit with a call without it: where the units of a batch fall on blocks, and so the order of the
    # sums, depends on all of its requests.)
    want, _, tol = ref.attention(q, cache.codes.cpu(), cache.meta.cpu(), table, kv, cu.tolist(), D ** -0.5, True)

    def first_only(out):
        return ((out[0] - want[0]).abs() <= tol[0]).all() and (out[1:] == 77).all()

    for l, c in ((i32([300, table.shape[1] * page + 1]), cu), (i32([300, -1]), cu), (lens, i32([0, 1, 4])),
                 (lens, i32([0, 1, 0])), (lens, i32([0, 1, 2 ** 31 - 1]))):
        assert first_only(run(table, l, c))
    out = run(table, lens, i32([-1, 1, 3]))
    assert (out[0] == 77).all() and ((out[1:] - want[1:]).abs() <= tol[1:]).all()
    assert first_only(run(table, lens, cu, max_q=1))  # the second request brings two


def test_attention_in_a_graph_with_lengths_that_grow(dev):
    Hq, H, D, page, B = 8, 2, 128, 16, 3
    cache = mx.kv4_cache(64, H, D, page, dev)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    lens, new, status = i32([0, 0, 0]), i32([1, 1, 1]), i32([0])
    table = torch.full((B, 20), -1, dtype=torch.int32, device=dev)
    free, count = torch.randperm(64, device=dev).to(torch.int32), i32([64])
    cu, slots, pos = i32([0] * 4), torch.zeros(4, dtype=torch.int64, device=dev), i32([0] * 4)
    x = torch.randn((4, Hq + 2 * H, D), device=dev).half()
    rope, q = mx.rope_table(512, D, device=dev), torch.zeros((4, Hq, D), dtype=torch.float16, device=dev)
    out = torch.zeros_like(q)
    ws = mx.kv4_attention_workspace(B, 1, Hq, cache, 20)

    def step():
        mx.kv4_assign_into(lens, new, table, free, count, page, lens, cu, slots, pos, count, status)
        mx.kv4_append_into(x[:, Hq:Hq + H], x[:, Hq + H:], slots, cache, q=x[:, :Hq], q_out=q, positions=pos, rope=rope)
        mx.kv4_attention_into(q, cache, table, lens, cu, 1, out, ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(40):
        x.normal_()
        new.copy_(i32([1, i % 2, 0 if i % 3 else 1]))
        graph.replay()
    mx.sync_status()
    assert int(status) == 0
    n = int(cu[-1])
    want, _, tol = ref.attention(q.cpu(), cache.codes.cpu(), cache.meta.cpu(), table.cpu(), lens.tolist(), cu.tolist(),
                                 D ** -0.5, True)
    assert ((out[:n].cpu().double() - want[:n]).abs() <= tol[:n]).all()
    assert lens.tolist()[0] == 41
    used = [-(-v // page) for v in lens.tolist()]
    pages = [int(table[b, j]) for b in range(B) for j in range(used[b])]
    assert len(set(pages)) == len(pages) and int(count) == 64 - len(pages)


def test_two_streams_with_their_own_workspaces(dev):
    a = _case(dev, [3000, 2000], [1, 1], 8, 2, 128, 64, seed=1)
    b = _case(dev, [1500, 2500], [1, 1], 8, 2, 128, 64, seed=2)
    alone = [mx.kv4_attention(c[0].to(dev), c[1], c[2].to(dev), c[3], c[4], 1) for c in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    held = [(c[0].to(dev), c[1], c[2].to(dev), c[3], c[4], 1, torch.zeros_like(alone[0]),
             mx.kv4_attention_workspace(2, 1, 8, c[1], c[2].shape[1])) for c in (a, b)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, h in zip(streams, held):
            mx.kv4_attention_into(*h, stream=s)
    torch.cuda.synchronize()
    mx.sync_status()
    for h, want in zip(held, alone):
        assert torch.equal(h[6], want)


def _within(dev, out, case, causal=True):
    q, cache, table, lens, cu = case
    D = q.shape[2]
    want, _, tol = ref.attention(q, cache.codes.cpu(), cache.meta.cpu(), table, lens.tolist(), cu.tolist(), D ** -0.5, causal)
    n = int(cu[-1])
    return bool(((out[:n].cpu().double() - want[:n]).abs() <= tol[:n]).all())


def test_one_workspace_serves_calls_of_all_sizes(dev):
    cases = [_case(dev, kv, qs, Hq, H, D, 64, seed=i) for i, (kv, qs, Hq, H, D) in enumerate([
        ([3000, 10], [1, 1], 8, 2, 128), ([400, 300], [100, 33], 4, 1, 128), ([900], [1], 4, 4, 64),
        ([700, 5, 90], [4, 2, 1], 6, 2, 64), ([2000], [9], 8, 2, 64)])]
    need = [mx.kv4_attention_workspace(len(c[3]), int(c[4].diff().max()), c[0].shape[1], c[1], c[2].shape[1]).numel()
            for c in cases]
    ws = torch.zeros(max(need), dtype=torch.uint8, device=dev)
    for _ in range(3):
        for c in cases:
            out = mx.kv4_attention(c[0].to(dev), c[1], c[2].to(dev), c[3], c[4], int(c[4].diff().max()), workspace=ws)
            assert _within(dev, out, c)
            assert not ws[:4096].any()
    mx.sync_status()


def test_prompts_in_a_graph_with_other_lengths(dev):
    """One captured call, replayed for lengths from nothing to the most it was captured for."""
    Hq, H, D, page = 4, 2, 128, 64
    full = _case(dev, [600, 500, 300], [200, 90, 300], Hq, H, D, page, seed=3)
    q, cache, table, lens, cu = full
    qd, td = q.to(dev), table.to(dev)
    out = torch.zeros_like(qd)
    ws = mx.kv4_attention_workspace(3, 300, Hq, cache, table.shape[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mx.kv4_attention_into(qd, cache, td, lens, cu, 300, out, ws, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.kv4_attention_into(qd, cache, td, lens, cu, 300, out, ws)
    for kv, qs in (([600, 500, 300], [200, 90, 300]), ([600, 1, 300], [1, 1, 17]), ([0, 0, 0], [0, 0, 0]),
                   ([128, 129, 0], [128, 0, 2]), ([600, 500, 300], [300, 300, 300])):
        lens.copy_(torch.tensor(kv, dtype=torch.int32))
        cu.copy_(torch.tensor([0, qs[0], qs[0] + qs[1], sum(qs)], dtype=torch.int32) if sum(qs) <= q.shape[0]
                 else torch.tensor([0, 290, 590, 590], dtype=torch.int32))
        out.fill_(77)
        graph.replay()
        mx.sync_status()
        assert _within(dev, out, (q, cache, table, lens, cu))
        assert (out[int(cu[-1]):] == 77).all()


def test_attention_of_nothing(dev):
    cache = mx.kv4_cache(2, 2, 64, 16, dev)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    q = torch.zeros((0, 4, 64), dtype=torch.float16, device=dev)
    assert mx.kv4_attention(q, cache, torch.zeros((0, 3), dtype=torch.int32, device=dev), i32([]), i32([0]), 0).numel() == 0
    assert mx.kv4_attention(q, cache, torch.zeros((2, 3), dtype=torch.int32, device=dev), i32([5, 0]), i32([0, 0, 0]), 1).numel() == 0
    q = torch.full((3, 4, 64), 1.0, dtype=torch.float16, device=dev)  # rows of no request
    out = mx.kv4_attention(q, cache, torch.zeros((1, 3), dtype=torch.int32, device=dev), i32([0]), i32([0, 0]), 3)
    assert not out.any()
    z = torch.zeros(0, dtype=torch.int64, device=dev)
    kv = torch.zeros((0, 2, 64), dtype=torch.float16, device=dev)
    mx.kv4_append_into(kv, kv, z, cache)
    mx.kv4_read_into(z, cache, kv, kv.clone())
    mx.sync_status()


def test_append_needs_what_goes_together(dev):
    cache = mx.kv4_cache(1, 1, 64, 16, dev)
    kv, slots = torch.zeros((2, 1, 64), dtype=torch.float16, device=dev), torch.arange(2, device=dev)
    with pytest.raises(ValueError, match="q_out"):
        mx.kv4_append_into(kv, kv, slots, cache, q=kv)
    with pytest.raises(ValueError, match="positions"):
        mx.kv4_append_into(kv, kv, slots, cache, rope=mx.rope_table(4, 64, device=dev))


def test_fresh_tensors_belong_to_the_given_stream(dev):
    """What kv4_attention and dequantize_act allocate is filled and reused in
    the given stream's order, however far behind the current one is."""
    H, D, page, T = 2, 64, 16, 1000
    cache = mx.kv4_cache(64, H, D, page, dev)
    kv = torch.randn((T, 2 * H, D), device=dev).half()
    mx.kv4_append_into(kv[:, :H], kv[:, H:], torch.arange(T, device=dev), cache)
    table = torch.arange(64, dtype=torch.int32, device=dev).reshape(1, 64)
    seq = torch.tensor([T], dtype=torch.int32, device=dev)
    A_q, s_a = mx.quantize_act(torch.randn((64, 256), device=dev).half())
    back = mx.dequantize_act(A_q, s_a)
    s, big = torch.cuda.Stream(), torch.zeros(1 << 28, device=dev)
    for n in (1, 100):  # either kernel
        q = torch.randn((n, H, D), device=dev).half()
        cu = torch.tensor([0, n], dtype=torch.int32, device=dev)
        torch.full((1 << 22,), 255, dtype=torch.uint8, device=dev)  # freed: fresh memory need not be zero
        torch.cuda.synchronize()
        for _ in range(10):
            big.add_(1)  # the current stream is busy
        out = mx.kv4_attention(q, cache, table, seq, cu, n, stream=s)
        X = mx.dequantize_act(A_q, s_a, stream=s)
        for _ in range(10):
            big.add_(1)
        torch.cuda.synchronize()
        mx.sync_status()
        assert _within(dev, out, (q.cpu(), cache, table.cpu(), seq, cu))
        assert torch.equal(X, back)


def test_everything_on_a_stream_of_its_own(dev):
    """The given stream orders the calls, whatever the current one does."""
    H, D, page, T = 2, 64, 16, 40
    cache = mx.kv4_cache(8, H, D, page, dev)
    x = torch.randn((T, 3 * H, D), device=dev).half()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    ctx, new, table = i32([0]), i32([T]), torch.full((1, 4), -1, dtype=torch.int32, device=dev)
    free, count, seq, cu = i32(list(range(8))), i32([8]), i32([0]), i32([0, 0])
    slots, pos = torch.zeros(T, dtype=torch.int64, device=dev), torch.zeros(T, dtype=torch.int32, device=dev)
    left, status, rope = i32([0]), i32([-1]), mx.rope_table(64, D, device=dev)
    q, out = torch.zeros((T, H, D), dtype=torch.float16, device=dev), torch.zeros((T, H, D), dtype=torch.float16, device=dev)
    ws = mx.kv4_attention_workspace(1, T, H, cache, 4)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    big = torch.zeros(1 << 28, device=dev)
    big.add_(1)  # the current stream is busy
    for _ in range(3):
        mx.kv4_assign_into(ctx, new, table, free, count, page, seq, cu, slots, pos, left, status, stream=s)
        mx.kv4_append_into(x[:, H:2 * H], x[:, 2 * H:], slots, cache, q=x[:, :H], q_out=q, positions=pos, rope=rope, stream=s)
        mx.kv4_attention_into(q, cache, table, seq, cu, T, out, ws, stream=s)
    s.synchronize()
    mx.sync_status(s)
    assert int(status) == 0
    assert _within(dev, out, (q.cpu(), cache, table.cpu(), seq, cu))
