"""Attention over the 4-bit cache where value scales differ by orders of
magnitude: a row's result depends on the tokens that it sees and gives weight
to, whatever scales the other tokens have.  GPU only."""
import pytest

torch = pytest.importorskip("torch")

import mixed_precision_quantized_act_b200 as mx  # noqa: E402
from tests import kv4_exact  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.load()
    return torch.device("cuda:0")


def _cache(dev, kv, Hkv, D, page, seed, key_scale=0.1):
    """Requests of kv tokens with pages in random order; all value scales 2^-13."""
    g = torch.Generator().manual_seed(seed)
    used = [-(-n // page) for n in kv]
    pages = sum(used) + 1
    codes = torch.randint(0, 256, (pages, 2, Hkv, page, D // 2), generator=g, dtype=torch.uint8)
    z = torch.randint(0, 16, (pages, 2, Hkv, page), generator=g, dtype=torch.int32)
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(kv), max(used)), -1, dtype=torch.int32)
    for b, n in enumerate(used):
        table[b, :n] = order[sum(used[:b]):sum(used[:b + 1])]
    scale = torch.full((pages, 2, Hkv, page), 2.0 ** -13)
    scale[:, 0] = key_scale
    return codes, z, scale, table, g


def _handle(dev, codes, z, scale):
    meta = (scale.half().view(torch.int16).to(torch.int32) & 0xFFFF) | z << 16
    return mx.KV4Cache(codes.to(dev), meta.to(dev))


def _run(dev, q, cache, table, kv, qs, causal=True, scale=None):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    cu = [sum(qs[:i]) for i in range(len(qs) + 1)]
    lens, cu, max_q, D = i32(kv), i32(cu), max(qs), q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    q = q.to(dev)
    out = torch.full_like(q, 77.0)
    lse = torch.full(q.shape[:2], 77.0, device=dev)
    ws = mx.kv4_attention_workspace(len(kv), max_q, q.shape[1], cache, table.shape[1])
    mx.kv4_attention_into(q, cache, table.to(dev), lens, cu, max_q, out, ws, scale, causal, lse)
    mx.sync_status()
    want, want_lse, tol, lse_tol = kv4_exact.attention(q, cache, table.to(dev), lens, cu, scale, causal)
    return kv4_exact.off_by(out, want, tol), kv4_exact.off_by(lse, want_lse, lse_tol)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,n,context", [(2, 1, 2, 0), (4, 2, 4, 0), (8, 1, 2, 300),          # few rows
                                              (4, 1, 70, 0), (2, 2, 150, 0), (3, 1, 100, 200)])   # prompts
@pytest.mark.parametrize("power", [12, 4])
def test_tokens_that_are_not_seen_yet_have_no_say(dev, D, Hq, Hkv, n, context, power):
    """The newest tokens' values are 2^17 or 2^25 times as large as those before:
    queries that come earlier do not see them."""
    kv, page = [context + n], 16
    codes, z, scale, table, g = _cache(dev, kv, Hkv, D, page, seed=D + n + power)
    for t in range(context + n - max(1, n // 2), context + n):
        scale[table[0, t // page].long(), 1, :, t % page] = 2.0 ** power
    q = torch.randn((n, Hq, D), generator=g).half()
    off = _run(dev, q, _handle(dev, codes, z, scale), table, kv, [n])
    assert max(off) <= 1, off


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,n", [(2, 1, 1), (4, 1, 4), (4, 1, 90)])
@pytest.mark.parametrize("where", [0, 40, 399])
def test_tokens_without_weight_have_no_say(dev, D, Hq, Hkv, n, where):
    """One token has values 2^25 times as large as the others' and a score at
    least 60 powers of two below theirs."""
    kv, page = [400], 16
    codes, z, scale, table, g = _cache(dev, kv, Hkv, D, page, seed=D + n + where)
    at = (table[0, where // page].long(), slice(None), where % page)
    codes[at[0], 0, :, at[2]] = 0
    z[at[0], 0, :, at[2]] = 15                         # key: -15 s in every channel
    # queries with a positive mean: sum q = D / 4 at least
    q = (torch.rand((n, Hq, D), generator=g) * 0.5 + 0.25).half()
    scale[at[0], 0, :, at[2]] = 60 * 0.6931 / (15 * D / 4 * D ** -0.5)
    scale[at[0], 1, :, at[2]] = 2.0 ** 12
    off = _run(dev, q, _handle(dev, codes, z, scale), table, kv, [n], causal=False)
    assert max(off) <= 1, off


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,n", [(2, 1, 1), (4, 1, 4), (4, 1, 90)])
def test_value_rows_of_zeros_take_their_share(dev, D, Hq, Hkv, n):
    """A token whose values are all zero (a scale of zero) has nearly all the
    weight: the others' share of the result is what the denominator leaves."""
    kv, page = [300], 32
    codes, z, scale, table, g = _cache(dev, kv, Hkv, D, page, seed=D + n)
    scale[:, 1] = 0.5
    q = (torch.rand((n, Hq, D), generator=g) * 0.5 + 0.25).half()
    for where, power in ((7, 3), (290, 8), (290, 60)):
        row = (table[0, where // page].long(), slice(None), where % page)
        codes[row[0], 0, :, row[2]] = 255
        z[row[0], 0, :, row[2]] = 0                    # key: 15 s in every channel
        scale[row[0], 0, :, row[2]] = power * 0.6931 / (15 * D / 4 * D ** -0.5)
        scale[row[0], 1, :, row[2]] = 0
        off = _run(dev, q, _handle(dev, codes, z, scale), table, kv, [n], causal=False)
        assert max(off) <= 1, (where, off)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 4, 90])
@pytest.mark.parametrize("causal", [True, False])
def test_value_scales_of_all_sizes_in_any_order(dev, D, n, causal):
    kv, qs, page, Hq, Hkv = [700, 130], [n, min(n, 3)], 64, 4, 2
    codes, z, scale, table, g = _cache(dev, kv, Hkv, D, page, seed=3 * D + n, key_scale=0.3)
    scale[:, 1] = torch.exp2(torch.rand(scale[:, 1].shape, generator=g) * 36 - 24)
    scale[:, 1][torch.rand(scale[:, 1].shape, generator=g) < 0.1] = 0
    q = torch.randn((sum(qs), Hq, D), generator=g).half()
    off = _run(dev, q, _handle(dev, codes, z, scale), table, kv, qs, causal)
    assert max(off) <= 1, off
