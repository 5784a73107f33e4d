"""The KV-cache operators on caches beyond 2^32 bytes, on pages that requests
share, and on two streams at once.  GPU only."""
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


def _i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


@pytest.mark.parametrize("n", [1, 130])  # either attention kernel
def test_pages_behind_the_first_4_gib(dev, n):
    """The same rows in a small cache and at the end of one of 4.4 GiB."""
    H, Hq, D, page, kv = 8, 16, 128, 64, 700
    used = -(-kv // page)
    pages = 2 ** 32 // (2 * H * page * D // 2) + 6000
    big = mx.KV4Cache(torch.empty((pages, 2, H, page, D // 2), dtype=torch.uint8, device=dev),
                      torch.empty((pages, 2, H, page), dtype=torch.int32, device=dev))
    assert big.codes.numel() > 2 ** 32
    small = mx.kv4_cache(used, H, D, page, dev)
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn((kv, 2 * H, D), generator=g, device=dev).half()
    q = torch.randn((n, Hq, D), generator=g, device=dev).half()
    at = torch.arange(kv, device=dev)
    outs = []
    for cache, first in ((small, 0), (big, pages - used)):
        slots = at + first * page
        mx.kv4_append_into(x[:, :H], x[:, H:], slots, cache)
        k, v = torch.zeros((kv, H, D), dtype=torch.float16, device=dev), torch.zeros((kv, H, D), dtype=torch.float16, device=dev)
        mx.kv4_read_into(slots, cache, k, v)
        table = torch.arange(first, first + used, dtype=torch.int32, device=dev).view(1, -1)
        out = mx.kv4_attention(q, cache, table, _i32([kv], dev), _i32([0, n], dev), n)
        mx.sync_status()
        outs.append((k, v, out))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 4, 60])
def test_requests_that_share_pages(dev, D, n):
    """A common prefix held once, in the tables of all requests."""
    B, H, Hq, page, prefix, kv = 5, 2, 8, 16, 800, [800 + n, 830 + n, 801 + n, 1000 + n, 800 + n]
    g = torch.Generator(device="cuda").manual_seed(D + n)
    own = [-(-(k - prefix) // page) for k in kv]
    pages = prefix // page + sum(own)
    codes = torch.randint(0, 256, (pages, 2, H, page, D // 2), generator=g, device=dev, dtype=torch.uint8)
    s = (torch.rand((pages, 2, H, page), generator=g, device=dev) * 0.3 + 0.05).half()
    z = torch.randint(0, 16, s.shape, generator=g, device=dev, dtype=torch.int32)
    cache = mx.KV4Cache(codes, (s.view(torch.int16).to(torch.int32) & 0xFFFF) | z << 16)
    table = torch.full((B, prefix // page + max(own)), -1, dtype=torch.int32, device=dev)
    table[:, :prefix // page] = torch.arange(prefix // page, dtype=torch.int32, device=dev)
    for b in range(B):
        first = prefix // page + sum(own[:b])
        table[b, prefix // page:prefix // page + own[b]] = torch.arange(first, first + own[b], dtype=torch.int32, device=dev)
    q = torch.randn((B * n, Hq, D), generator=g, device=dev).half()
    lens, cu = _i32(kv, dev), _i32([n * i for i in range(B + 1)], dev)
    out = mx.kv4_attention(q, cache, table, lens, cu, n)
    mx.sync_status()
    want, _, tol, _ = kv4_exact.attention(q, cache, table, lens, cu, D ** -0.5)
    assert kv4_exact.off_by(out, want, tol) <= 1


def test_a_prompt_and_a_decode_step_on_two_streams(dev):
    """Calls that overlap, with workspaces of their own, over one cache."""
    H, Hq, D, page, kv = 4, 16, 128, 64, 3000
    pages = 2 * -(-kv // page)
    cache = mx.kv4_cache(pages, H, D, page, dev)
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn((pages * page, 2 * H, D), generator=g, device=dev).half()
    mx.kv4_append_into(x[:, :H], x[:, H:], torch.arange(pages * page, device=dev), cache)
    table = torch.randperm(pages, generator=g, device=dev).to(torch.int32).view(2, -1)
    lens = _i32([kv, kv - 100], dev)
    calls = []
    for n in (300, 1):
        q = torch.randn((2 * n, Hq, D), generator=g, device=dev).half()
        cu = _i32([0, n, 2 * n], dev)
        want = mx.kv4_attention(q, cache, table, lens, cu, n)
        calls.append((want, (q, cache, table, lens, cu, n, torch.zeros_like(q),
                             mx.kv4_attention_workspace(2, n, Hq, cache, table.shape[1]))))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for stream, (_, args) in zip(streams, calls):
            mx.kv4_attention_into(*args, stream=stream)
    torch.cuda.synchronize()
    mx.sync_status()
    for want, args in calls:
        assert torch.equal(args[6], want)
