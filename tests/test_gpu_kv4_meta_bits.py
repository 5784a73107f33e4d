"""Bits of a cache's metadata words above the zero point mean nothing.  GPU only."""
import pytest

torch = pytest.importorskip("torch")

import mixed_precision_quantized_act_b200 as mx  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 3, 70])  # one and two 8-row tiles, prompts
def test_bits_above_the_zero_point_are_not_read(D, n):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev, H, Hq, page, kv = torch.device("cuda:0"), 2, 8, 16, 300
    g = torch.Generator(device="cuda").manual_seed(D + n)
    pages = -(-kv // page)
    codes = torch.randint(0, 256, (pages, 2, H, page, D // 2), generator=g, device=dev, dtype=torch.uint8)
    s = (torch.rand((pages, 2, H, page), generator=g, device=dev) * 0.3 + 0.05).half()
    z = torch.randint(0, 16, s.shape, generator=g, device=dev, dtype=torch.int32)
    meta = (s.view(torch.int16).to(torch.int32) & 0xFFFF) | z << 16
    above = torch.randint(0, 1 << 12, s.shape, generator=g, device=dev, dtype=torch.int32) << 20
    q = torch.randn((n, Hq, D), generator=g, device=dev).half()
    table = torch.arange(pages, dtype=torch.int32, device=dev).view(1, -1)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    want, got = (mx.kv4_attention(q, mx.KV4Cache(codes, m), table, i32([kv]), i32([0, n]), n) for m in (meta, meta | above))
    mx.sync_status()
    assert want.isfinite().all() and torch.equal(got, want)
