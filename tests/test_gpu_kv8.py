"""The paged 8-bit KV cache on the GPU: append, read-back and attention against
plain restatements of their definitions.  GPU only."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mixed_precision_quantized_act_b200 as mx  # noqa: E402
from mixed_precision_quantized_act_b200 import _lib  # noqa: E402
from tests import kv4_ref  # noqa: E402
from tests import kv8_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.load()
    return torch.device("cuda:0")


def _gen(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


def _filled(dev, pages, H, D, page, seed=0, wide=False):
    """A cache of codes spread like those of normal values and scales within a factor of 3 (wide: of 10^6)."""
    g = _gen(dev, seed)
    shape = (pages, 2, H, page, D)
    codes = (torch.randn(shape, generator=g, device=dev) * 40).round().clamp(-127, 127).add(128).to(torch.uint8)
    u = torch.rand(shape[:3] + (page // 16,), generator=g, device=dev)
    return mx.KV8Cache(codes, 10.0 ** (-6 * u) if wide else 0.01 + 0.02 * u)


# ------------------------------------------------------------------ append and read

def _slots(lens, page, g, dev):
    """Slots of requests' tokens [old, old + new) in pages of their own, as kv4_assign lists them, and the pages."""
    used = [-(-(old + new) // page) for old, new in lens]
    order = torch.randperm(sum(used) + 1, generator=g, device=dev)
    out, at = [], 0
    for (old, new), n in zip(lens, used):
        row = torch.arange(old, old + new, device=dev)
        out.append(order[at + row // page] * page + row % page)
        at += n
    return torch.cat(out), sum(used) + 1


def _check_append(dev, lens, H, D, page, seed=0, scale=1.0):
    g = _gen(dev, seed)
    slots, pages = _slots(lens, page, g, dev)
    T = slots.numel()
    cache = _filled(dev, pages, H, D, page, seed)
    codes, scales = cache.codes.cpu().numpy(), cache.scales.cpu().numpy()
    kv = (torch.randn((T, 2 * H, D), generator=g, device=dev) * scale).half()
    mx.kv8_append_into(kv[:, :H], kv[:, H:], slots, cache)
    mx.sync_status()
    host = kv.cpu().numpy()
    codes, scales = ref.append(codes, scales, slots.tolist(), host[:, :H], host[:, H:])
    assert np.array_equal(cache.scales.cpu().numpy().view(np.uint32), scales.view(np.uint32))
    assert np.array_equal(cache.codes.cpu().numpy(), codes)
    return cache, slots, kv


@pytest.mark.parametrize("lens", [[(0, 1)], [(5, 1)], [(15, 1), (16, 1), (0, 1), (31, 2)], [(0, 16)], [(3, 40), (0, 0), (7, 9)],
                                  [(9, 700), (0, 33)], [(i % 16, 1) for i in range(100)], [(1, 1)] * 600], ids=str)
@pytest.mark.parametrize("H,D,page", [(2, 128, 16), (3, 64, 64), (1, 128, 256)])
def test_append_writes_the_definition(dev, lens, H, D, page):
    """Blocks that begin, end and grow within a call, against numpy, bit for bit; small values leave older scales."""
    for scale in (3.0, 0.05):
        _check_append(dev, lens, H, D, page, seed=len(lens), scale=scale)


def test_blocks_that_grow_step_by_step(dev):
    """One token at a time, each larger than the last: every older row is coded again, as the definition says."""
    H, D, page = 2, 64, 16
    cache = _filled(dev, 2, H, D, page)
    codes, scales = cache.codes.cpu().numpy(), cache.scales.cpu().numpy()
    for t in range(20):
        kv = (torch.randn((1, 2 * H, D), generator=_gen(dev, t), device=dev) * 1.3 ** t).half()
        slot = torch.tensor([t], device=dev)
        mx.kv8_append_into(kv[:, :H], kv[:, H:], slot, cache)
        host = kv.cpu().numpy()
        codes, scales = ref.append(codes, scales, [t], host[:, :H], host[:, H:])
        assert np.array_equal(cache.codes.cpu().numpy(), codes) and np.array_equal(cache.scales.cpu().numpy(), scales)
    mx.sync_status()


@pytest.mark.parametrize("H,D,page", [(2, 128, 64), (1, 64, 16)])
def test_read_back(dev, H, D, page):
    cache = _filled(dev, 7, H, D, page, 1)
    cache.scales[0, 0, 0, 0] = 600.0  # beyond the largest fp16
    slots = torch.randperm(7 * page, device=dev)[:90]
    slots[0], slots[3] = 2, -1
    k, v = (torch.full((90, H, D), 77.0, dtype=torch.float16, device=dev) for _ in range(2))
    mx.kv8_read_into(slots, cache, k, v)
    mx.sync_status()
    want = ref.values(cache.codes, cache.scales)[slots // page, :, :, slots % page].clamp(-65504, 65504)
    keep = slots >= 0
    assert torch.equal(k[keep], want[keep, 0].half()) and torch.equal(v[keep], want[keep, 1].half())
    assert (k[~keep] == 77).all() and (v[~keep] == 77).all()


@pytest.mark.parametrize("T", [5, 700])  # one kernel, and two
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("D,rotary", [(128, 128), (128, 32), (64, 64)])
def test_append_normalizes_and_rotates(dev, T, norm, D, rotary):
    """Queries and keys as head_norm_rope_into gives them, bit for bit, the keys then quantized."""
    Hq, H, page = 6, 2, 32
    g = _gen(dev, T + D)
    slots, pages = _slots([(3, T)], page, g, dev)
    x = torch.randn((T, Hq + 2 * H, D), generator=g, device=dev).half()
    w = [(1 + 0.2 * torch.randn(D, generator=g, device=dev)).half() for _ in range(2)] if norm else [None, None]
    pos = torch.randint(0, 300, (T,), generator=g, device=dev, dtype=torch.int32)
    rope = mx.rope_table(300, rotary, device=dev)
    q, k, v = x.split((Hq, H, H), 1)
    want_q, want_k = torch.empty((T, Hq, D), device=dev).half(), torch.empty((T, H, D), device=dev).half()
    mx.head_norm_rope_into(q, want_q, w[0], k=k, k_out=want_k, w_k=w[1], positions=pos, rope=rope, eps=1e-5)
    if not norm:
        rot = kv4_ref.rotate(k.cpu().numpy(), rope.cpu().numpy(), pos.cpu().numpy(), rotary)
        assert np.array_equal(want_k.cpu().numpy().view(np.uint16), rot.view(np.uint16))
    cache = _filled(dev, pages, H, D, page)
    codes, scales = cache.codes.cpu().numpy(), cache.scales.cpu().numpy()
    out = torch.full_like(want_q, 77.0)
    mx.kv8_append_into(k, v, slots, cache, q=q, q_out=out, positions=pos, rope=rope, w_q=w[0], w_k=w[1], eps=1e-5)
    mx.sync_status()
    assert torch.equal(out, want_q)
    codes, scales = ref.append(codes, scales, slots.tolist(), want_k.cpu().numpy(), v.cpu().numpy())
    assert np.array_equal(cache.scales.cpu().numpy(), scales) and np.array_equal(cache.codes.cpu().numpy(), codes)
    # in place, into the same slots: nothing grows any more, the codes stay
    mx.kv8_append_into(k, v, slots, cache, q=q, q_out=q, positions=pos, rope=rope, w_q=w[0], w_k=w[1], eps=1e-5)
    mx.sync_status()
    assert torch.equal(x[:, :Hq], want_q) and np.array_equal(cache.codes.cpu().numpy(), codes)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("kind", [0, 1])
def test_what_is_not_finite_stays_in_its_block(dev, bad, kind):
    H, D, page = 2, 128, 32
    cache = mx.kv8_cache(2, H, D, page, dev)
    kv = torch.randn((40, 2, H, D), device=dev).half()
    kv[20, kind, 1, 77] = bad
    slots = torch.arange(40, device=dev)
    mx.kv8_append_into(kv[:, 0], kv[:, 1], slots, cache)
    assert cache.scales.isnan().nonzero().tolist() == [[0, kind, 1, 1]]
    out = [torch.empty((40, H, D), dtype=torch.float16, device=dev) for _ in range(2)]
    mx.kv8_read_into(slots, cache, *out)
    assert out[kind][16:32, 1].isnan().all() and out[kind][:16].isfinite().all() and out[kind][32:].isfinite().all()
    assert out[1 - kind].isfinite().all() and out[kind][:, 0].isfinite().all()
    one = torch.ones((1, H, D), device=dev).half()
    mx.kv8_append_into(one, one, slots[21:22], cache)  # it stays
    assert bool(cache.scales[0, kind, 1, 1].isnan())
    mx.kv8_append_into(one, one, slots[16:17], cache)  # until the block begins anew
    mx.sync_status()
    assert cache.scales.isfinite().all()


def test_rows_of_zeros(dev):
    cache = _filled(dev, 1, 1, 64, 16)
    z = torch.zeros((16, 1, 64), dtype=torch.float16, device=dev)
    mx.kv8_append_into(z, z, torch.arange(16, device=dev), cache)
    mx.sync_status()
    assert (cache.scales == 0).all() and (cache.codes == 128).all()
    z[3] = 1
    mx.kv8_append_into(z[3:4], z[3:4], torch.tensor([3], device=dev), cache)
    assert (cache.codes[0, :, 0, 3] == 255).all() and (cache.codes[0, :, 0, :3] == 128).all()


@pytest.mark.parametrize("T", [40, 800])
def test_slots_and_positions_out_of_range_are_reported(dev, T):
    Hq, H, D, page = 3, 2, 64, 16
    g = _gen(dev, T)
    x = torch.randn((T, Hq + 2 * H, D), generator=g, device=dev).half()
    q, k, v = x.split((Hq, H, H), 1)
    rope = mx.rope_table(T + 5, D, device=dev)
    good = torch.arange(T, device=dev) + 16
    pos = torch.arange(T, dtype=torch.int32, device=dev)

    def run(slots, pos):
        cache = _filled(dev, T // 16 + 3, H, D, page, 5)
        out = torch.full((T, Hq, D), 77.0, dtype=torch.float16, device=dev)
        mx.kv8_append_into(k, v, slots, cache, q=q, q_out=out, positions=pos, rope=rope)
        return cache, out

    clean, want = run(good, pos)
    mx.sync_status()
    skipped = good.clone()
    skipped[16:32] = -1  # a block's tokens: no error
    cache, out = run(skipped, pos)
    mx.sync_status()
    assert (out[16:32] == 77).all() and torch.equal(out[:16], want[:16]) and torch.equal(out[32:], want[32:])
    untouched = _filled(dev, T // 16 + 3, H, D, page, 5)
    assert torch.equal(cache.codes[2], untouched.codes[2]) and torch.equal(cache.scales[2], untouched.scales[2])
    assert torch.equal(cache.codes[[1, 3]], clean.codes[[1, 3]])
    for wrong in ("slot", "position below", "position beyond"):
        s, p = good.clone(), pos.clone()
        if wrong == "slot":
            s[16:32] = (T // 16 + 3) * page + torch.arange(16, device=dev)
        else:
            p[16:32] = -1 if wrong == "position below" else T + 5
        cache, out = run(s, p)
        with pytest.raises(_lib.MixLLMError) as e:
            mx.sync_status()
        assert e.value.status == _lib.ERR_BOUNDS
        assert (out[16:32] == 77).all() and torch.equal(out[32:], want[32:])
        assert torch.equal(cache.codes[2], untouched.codes[2]) and torch.equal(cache.codes[[1, 3]], clean.codes[[1, 3]])


# ------------------------------------------------------------------ attention

def _case(dev, kv, qs, Hq, H, D, page, seed=0, wide=False):
    g = _gen(dev, seed)
    used = [-(-n // page) for n in kv]
    W, pages = max(used + [1]), sum(used) + 2
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32).cpu()
    table, at = torch.full((len(kv), W), -1, dtype=torch.int32), 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    cache = _filled(dev, pages, H, D, page, seed, wide)
    q = torch.randn((sum(qs) + 0, Hq, D), generator=g, device=dev).half().cpu()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    return q, cache, table, i32(kv), i32([sum(qs[:i]) for i in range(len(qs) + 1)])


def _check(dev, kv, qs, Hq, H, D, page, causal=True, scale=None, seed=0, wide=False, tail=0):
    q, cache, table, lens, cu = _case(dev, kv, qs, Hq, H, D, page, seed, wide)
    q = torch.cat((q, torch.ones((tail, Hq, D), dtype=torch.float16)))
    scale = D ** -0.5 if scale is None else scale
    # what lies behind a request's last token is of no meaning: blocks of NaN scales, codes of anything
    for b, n in enumerate(kv):
        if n % page:
            p = int(table[b, n // page])
            cache.codes[p, :, :, n % page:] = torch.randint(0, 256, cache.codes[p, :, :, n % page:].shape, device=dev).to(torch.uint8)
            cache.scales[p, :, :, -(-(n % page) // 16):] = float("nan")
    out = torch.full(q.shape, 77.0, dtype=torch.float16, device=dev)
    lse = torch.full(q.shape[:2], 77.0, device=dev)
    ws = mx.kv8_attention_workspace(len(kv), max(qs), Hq, cache, table.shape[1])
    args = (q.to(dev), cache, table.to(dev), lens, cu, max(qs))
    mx.kv8_attention_into(*args, out, ws, scale, causal, lse)
    mx.sync_status()
    want, want_lse, tol = ref.attention(q, cache.codes.cpu(), cache.scales.cpu().nan_to_num(0.0), table, kv, cu.tolist(),
                                        scale, causal)
    n = int(cu[-1])
    off = (out.cpu().double()[:n] - want[:n]).abs()
    assert (off <= tol[:n]).all(), (float((off / tol[:n].clamp(min=1e-30)).max()), float(off.max()))
    assert (out[n:] == 77).all() and (lse[n:] == 77).all()
    seen = want_lse[:n] > -float("inf")
    assert (lse[:n].cpu()[~seen] == -float("inf")).all()
    far = (lse[:n].cpu().double() - want_lse[:n]).abs()[seen]
    # the relative errors of the probabilities' sum (the tolerance's e), and the rounding of the result
    assert (far <= 2.0 ** -18 * (1 + want_lse[:n].abs()[seen]) + 64 * D * 2.0 ** -24).all()
    again = torch.full_like(out, 77.0)
    mx.kv8_attention_into(*args, again, ws, scale, causal)
    mx.sync_status()
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))
    assert not ws[:4096].any()


@pytest.mark.parametrize("kv", [[1], [0], [2, 15, 16, 17], [127, 128, 129, 130], [0, 300, 1, 0, 257], [4097, 1, 700]],
                         ids=str)
@pytest.mark.parametrize("Hq,H,D,page", [(8, 2, 128, 64), (4, 4, 64, 16), (8, 1, 128, 128), (6, 2, 64, 256),
                                         (2, 1, 128, 32)])
def test_attention_of_single_tokens(dev, kv, Hq, H, D, page):
    _check(dev, kv, [1] * len(kv), Hq, H, D, page, seed=len(kv))


@pytest.mark.parametrize("n", [16, 31, 255, 256, 257, 512, 513, 1003, 2048, 9001])
@pytest.mark.parametrize("Hq,H,D", [(4, 2, 128), (8, 8, 64)])
def test_attention_of_one_request(dev, n, Hq, H, D):
    """A single request's heads are cut alike: one block to a head, a few, all."""
    _check(dev, [n], [1], Hq, H, D, 64, seed=n)


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
    _check(dev, [9000, 4000], [40, 20], 1, 1, 128, 64, seed=7)


def test_attention_with_more_requests_than_threads(dev):
    kv = np.random.default_rng(1).integers(0, 60, 700).tolist()
    _check(dev, kv, [1] * 700, 2, 1, 64, 16, seed=7)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("qs", [[1, 2], [30, 20]], ids=str)
def test_attention_with_scales_of_all_sizes(dev, D, qs):
    _check(dev, [400, 129], qs, 4, 2, D, 64, seed=8, wide=True)


@pytest.mark.parametrize("scale", [1e-4, 3.0, -0.5])
@pytest.mark.parametrize("n", [1, 40])
def test_attention_with_other_scales(dev, scale, n):
    _check(dev, [333], [n], 4, 1, 128, 64, scale=scale, seed=9)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_a_block_scale_of_zero_is_a_value_of_zero(dev, n, D):
    """Whatever the codes: a cache that was never written holds none of 128 but zeros."""
    q, cache, table, lens, cu = _case(dev, [100], [n], 2, 1, D, 16, seed=2)
    cache.scales[table[0, 2], 1] = 0
    cache.codes[table[0, 2], 1] = 0
    cache.scales[table[0, 4], 0] = 0
    out = mx.kv8_attention(q.to(dev), cache, table.to(dev), lens, cu, n)
    mx.sync_status()
    want, _, tol = ref.attention(q, cache.codes.cpu(), cache.scales.cpu(), table, [100], cu.tolist(), D ** -0.5, True)
    assert ((out.cpu().double() - want).abs() <= tol).all()
    cache.scales[:, 1] = 0
    cache.codes[:, 1] = 7
    assert not mx.kv8_attention(q.to(dev), cache, table.to(dev), lens, cu, n).any()


@pytest.mark.parametrize("n", [1, 30])
def test_one_heavy_token_of_small_value_leaves_the_others(dev, n):
    """A token with nearly all the weight and a value near zero, in a block of its own scale: the rest decide."""
    D, page = 128, 16
    q, cache, table, lens, cu = _case(dev, [700], [n], 2, 1, D, page, seed=4)
    cache.scales[table[0, 0], 0] = 0.3
    cache.codes[table[0, 0], 0, :, 0] = (q[:, 0].float().mean(0).sign() * 100 + 128).to(torch.uint8).to(dev)
    cache.codes[table[0, 0], 0, :, 1:] = 128
    cache.scales[table[0, 0], 1] = 1e-7
    out = mx.kv8_attention(q.to(dev), cache, table.to(dev), lens, cu, n)
    mx.sync_status()
    want, _, tol = ref.attention(q, cache.codes.cpu(), cache.scales.cpu(), table, [700], cu.tolist(), D ** -0.5, True)
    assert ((out.cpu().double() - want).abs() <= tol).all()


def test_attention_takes_strided_tensors(dev):
    kv, qs, Hq, H, D, page = [150, 60], [2, 1], 4, 2, 128, 64
    q, cache, table, lens, cu = _case(dev, kv, qs, Hq, H, D, page)
    wide = torch.zeros((3, Hq + 2, D), dtype=torch.float16, device=dev)
    wide[:, 1:1 + Hq] = q.to(dev)
    out = torch.full((3, Hq + 3, D), 77.0, dtype=torch.float16, device=dev)
    big = torch.full((2, table.shape[1] + 5), -1, dtype=torch.int32, device=dev)
    big[:, :table.shape[1]] = table.to(dev)
    ws = mx.kv8_attention_workspace(2, 2, Hq, cache, table.shape[1])
    mx.kv8_attention_into(wide[:, 1:1 + Hq], cache, big[:, :table.shape[1]], lens, cu, 2, out[:, 2:2 + Hq], ws)
    want = mx.kv8_attention(q.to(dev), cache, table.to(dev), lens, cu, 2)
    mx.sync_status()
    assert torch.equal(out[:, 2:2 + Hq], want)
    assert (out[:, :2] == 77).all() and (out[:, 2 + Hq:] == 77).all()


@pytest.mark.parametrize("n", [3, 40])
def test_nan_blocks_poison_only_who_sees_them(dev, n):
    Hq, H, D, page = 4, 2, 128, 64
    q, cache, table, lens, cu = _case(dev, [208], [n], Hq, H, D, page)
    t = 207  # the last block, 192 .. 207
    for kind in (0, 1):
        scales = cache.scales.clone()
        scales[table[0, t // page], kind, 1, t % page // 16] = float("nan")
        out = mx.kv8_attention(q.to(dev), mx.KV8Cache(cache.codes, scales), table.to(dev), lens, cu, n)
        mx.sync_status()
        sees = torch.arange(n) + 208 - n >= 192
        assert out[~sees].isfinite().all() and out[:, :2].isfinite().all()
        assert out[sees][:, 2:].isnan().all()


def test_attention_reports_pages_and_lengths_out_of_range(dev):
    Hq, H, D, page = 4, 2, 128, 64
    for kv, qs in (([300, 100], [1, 2]), ([300, 100], [20, 30])):
        q, cache, table, lens, cu = _case(dev, kv, qs, Hq, H, D, page)

        def run(table, lens, cu, max_q):
            out = torch.full(q.shape, 77.0, dtype=torch.float16, device=dev)
            ws = mx.kv8_attention_workspace(2, max_q, Hq, cache, table.shape[1])
            mx.kv8_attention_into(q.to(dev), cache, table.to(dev), lens, cu, max_q, out, ws)
            with pytest.raises(_lib.MixLLMError) as e:
                mx.sync_status()
            assert e.value.status == _lib.ERR_BOUNDS
            assert not ws[:4096].any()
            return out.cpu().double()

        def want(t):
            return ref.attention(q, cache.codes.cpu(), cache.scales.cpu(), t, kv, cu.tolist(), D ** -0.5, True)

        for wrong in (-1, cache.pages, 2 ** 31 - 1, -2 ** 31):  # the tokens of a bad page are not seen
            bad = table.clone()
            bad[0, 2] = wrong
            o, _, tol = want(bad)
            assert ((run(bad, lens, cu, max(qs)) - o).abs() <= tol).all()
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
        o, _, tol = want(table)
        a, end = qs[0], sum(qs)
        for l, c in ((i32([300, table.shape[1] * page + 1]), cu), (i32([300, -1]), cu), (lens, i32([0, a, end + 1])),
                     (lens, i32([0, a, 0])), (lens, i32([0, a, 2 ** 31 - 1]))):
            got = run(table, l, c, max(qs))
            assert ((got[:a] - o[:a]).abs() <= tol[:a]).all() and (got[a:] == 77).all()


def test_append_and_attention_in_a_graph_with_lengths_that_grow(dev):
    Hq, H, D, page, B = 8, 2, 128, 16, 3
    cache = mx.kv8_cache(64, H, D, page, dev)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    lens, new, status = i32([0, 0, 0]), i32([1, 1, 1]), i32([0])
    table = torch.full((B, 20), -1, dtype=torch.int32, device=dev)
    free, count = torch.randperm(64, device=dev).to(torch.int32), i32([64])
    cu, slots, pos = i32([0] * 4), torch.zeros(4, dtype=torch.int64, device=dev), i32([0] * 4)
    x = torch.randn((4, Hq + 2 * H, D), device=dev).half()
    w = (1 + 0.1 * torch.randn((2, D), device=dev)).half()
    rope, q = mx.rope_table(512, D, device=dev), torch.zeros((4, Hq, D), dtype=torch.float16, device=dev)
    out = torch.zeros_like(q)
    ws = mx.kv8_attention_workspace(B, 1, Hq, cache, 20)

    def step():
        mx.kv4_assign_into(lens, new, table, free, count, page, lens, cu, slots, pos, count, status)
        mx.kv8_append_into(x[:, Hq:Hq + H], x[:, Hq + H:], slots, cache, q=x[:, :Hq], q_out=q, positions=pos, rope=rope,
                           w_q=w[0], w_k=w[1])
        mx.kv8_attention_into(q, cache, table, lens, cu, 1, out, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
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
    assert int(status) == 0 and lens.tolist()[0] == 41
    n = int(cu[-1])
    want, _, tol = ref.attention(q.cpu(), cache.codes.cpu(), cache.scales.cpu(), table.cpu(), lens.tolist(), cu.tolist(),
                                 D ** -0.5, True)
    assert ((out[:n].cpu().double() - want[:n]).abs() <= tol[:n]).all()


def _within(out, case):
    q, cache, table, lens, cu = case
    want, _, tol = ref.attention(q, cache.codes.cpu(), cache.scales.cpu(), table, lens.tolist(), cu.tolist(),
                                 q.shape[2] ** -0.5, True)
    return bool(((out.cpu().double() - want).abs() <= tol).all())


def test_one_workspace_serves_calls_of_all_sizes(dev):
    cases = [_case(dev, kv, qs, Hq, H, D, 64, seed=i) for i, (kv, qs, Hq, H, D) in enumerate([
        ([3000, 10], [1, 1], 8, 2, 128), ([400, 300], [100, 33], 4, 1, 128), ([900], [1], 4, 4, 64),
        ([700, 5, 90], [4, 2, 1], 6, 2, 64), ([2000], [9], 8, 2, 64)])]
    most = lambda c: int(c[4].diff().max())  # noqa: E731
    need = [mx.kv8_attention_workspace(len(c[3]), most(c), c[0].shape[1], c[1], c[2].shape[1]).numel() for c in cases]
    ws = torch.zeros(max(need), dtype=torch.uint8, device=dev)
    for _ in range(3):
        for c in cases:
            out = mx.kv8_attention(c[0].to(dev), c[1], c[2].to(dev), c[3], c[4], most(c), workspace=ws)
            assert _within(out, c)
            assert not ws[:4096].any()
    mx.sync_status()


def test_two_streams_with_their_own_workspaces(dev):
    cases = [_case(dev, kv, [1, 1], 8, 2, 128, 64, seed=i) for i, kv in enumerate(([3000, 2000], [1500, 2500]))]
    alone = [mx.kv8_attention(c[0].to(dev), c[1], c[2].to(dev), c[3], c[4], 1) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    held = [(c[0].to(dev), c[1], c[2].to(dev), c[3], c[4], 1, torch.zeros_like(alone[0]),
             mx.kv8_attention_workspace(2, 1, 8, c[1], c[2].shape[1])) for c in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, h in zip(streams, held):
            mx.kv8_attention_into(*h, stream=s)
    torch.cuda.synchronize()
    mx.sync_status()
    for h, want in zip(held, alone):
        assert torch.equal(h[6], want)


def test_slots_beyond_32_bits_of_bytes(dev):
    """A cache of more than 4 GB, whose last pages are written, read and attended."""
    H, D, page, pages = 8, 128, 256, 8300
    cache = mx.KV8Cache(torch.empty((pages, 2, H, page, D), dtype=torch.uint8, device=dev),
                        torch.zeros((pages, 2, H, page // 16), device=dev))
    assert cache.codes.numel() > 2 ** 32
    g = _gen(dev, 3)
    kv = torch.randn((300, 2 * H, D), generator=g, device=dev).half()
    slots = torch.cat((torch.arange(256, device=dev) + (pages - 1) * page, torch.arange(44, device=dev) + 8250 * page))
    mx.kv8_append_into(kv[:, :H], kv[:, H:], slots, cache)
    out = [torch.empty((300, H, D), dtype=torch.float16, device=dev) for _ in range(2)]
    mx.kv8_read_into(slots, cache, *out)
    for got, want in zip(out, (kv[:, :H], kv[:, H:])):
        step = want.float().abs().amax() / 127
        assert ((got.float() - want.float()).abs() <= step / 2 * 1.01 + 2.0 ** -11 * want.float().abs()).all()
    table = torch.tensor([[pages - 1, 8250]], dtype=torch.int32, device=dev)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    for n in (1, 20):
        q = torch.randn((n, H, D), generator=g, device=dev).half()
        att = mx.kv8_attention(q, cache, table, i32([300]), i32([0, n]), n)
        mx.sync_status()
        k, v = (x.double().transpose(0, 1) for x in out)
        sc = torch.einsum("ihd,htd->hit", q.double(), k) * D ** -0.5
        late = torch.arange(300, device=dev)[None, :] > 300 - n + torch.arange(n, device=dev)[:, None]
        want = torch.einsum("hit,htd->ihd", sc.masked_fill(late, -float("inf")).softmax(-1), v)
        # the values read back are rounded to fp16 once more: 2^-11 of each, in keys a score error of up to
        # 2^-11 sum |q k| scale (below 2^-11 * 128 * 4 * 4 / 11 < 0.1 here, in fact some sixteenth)
        assert ((att.double() - want).abs() <= 0.02 * (1 + want.abs())).all()


def test_nothing_to_do(dev):
    cache = mx.kv8_cache(2, 2, 64, 16, dev)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    q = torch.zeros((0, 4, 64), dtype=torch.float16, device=dev)
    assert mx.kv8_attention(q, cache, torch.zeros((0, 3), dtype=torch.int32, device=dev), i32([]), i32([0]), 0).numel() == 0
    q = torch.full((3, 4, 64), 1.0, dtype=torch.float16, device=dev)  # rows of no request
    assert not mx.kv8_attention(q, cache, torch.zeros((1, 3), dtype=torch.int32, device=dev), i32([0]), i32([0, 0]), 3).any()
    z, kv = torch.zeros(0, dtype=torch.int64, device=dev), torch.zeros((0, 2, 64), dtype=torch.float16, device=dev)
    mx.kv8_append_into(kv, kv, z, cache)
    mx.kv8_read_into(z, cache, kv, kv.clone())
    none = torch.full((40,), -1, dtype=torch.int64, device=dev)
    kv = torch.zeros((40, 2, 64), dtype=torch.float16, device=dev)
    mx.kv8_append_into(kv, kv, none, cache)
    mx.sync_status()
    assert (cache.codes == 128).all()


def test_bindings_check_their_tensors(dev):
    cache = mx.kv8_cache(2, 1, 64, 16, dev)
    kv, slots = torch.zeros((2, 1, 64), dtype=torch.float16, device=dev), torch.arange(2, device=dev)
    for bad in (lambda: mx.kv8_append_into(kv, kv, slots, cache, q=kv),
                lambda: mx.kv8_append_into(kv, kv, slots, cache, rope=mx.rope_table(4, 64, device=dev)),
                lambda: mx.kv8_append_into(kv, kv, slots, cache, w_k=kv[0]),
                lambda: mx.kv8_append_into(kv.float(), kv, slots, cache), lambda: mx.kv8_append_into(kv, kv, slots.int(), cache),
                lambda: mx.kv8_read_into(slots, cache, kv[:1], kv), lambda: mx.KV8Cache(cache.codes, cache.scales[:1]),
                lambda: mx.KV8Cache(cache.codes[0], cache.scales), lambda: mx.KV8Cache(cache.codes.int(), cache.scales)):
        with pytest.raises(ValueError):
            bad()
