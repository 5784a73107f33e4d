"""layer.AttentionBlock on a stream other than the one it was constructed on:
its buffers are filled by the time the constructor returns.  GPU only."""
import pytest

torch = pytest.importorskip("torch")

import mixed_precision_quantized_act_b200 as mx  # noqa: E402
from mixed_precision_quantized_act_b200.layer import AttentionBlock  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 100])
def test_a_fresh_block_runs_on_any_stream(tokens):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev = torch.device("cuda:0")
    Hq, H, D, K, page, context = 8, 2, 64, 256, 16, 2000
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    qkv = mx.pack_weights(rand((Hq + 2 * H) * D, K) * 0.06, torch.zeros((Hq + 2 * H) * D, dtype=torch.uint8, device=dev))
    o = mx.pack_weights(rand(K, Hq * D) * 0.06, torch.zeros(K, dtype=torch.uint8, device=dev))
    w, r = torch.ones(K, dtype=torch.float16, device=dev), rand(tokens, K)
    pages = -(-(context + tokens) // page)
    old = rand(context, 2 * H, D).half()
    table = torch.arange(pages, dtype=torch.int32, device=dev).view(1, -1)
    lens = torch.tensor([context + tokens], dtype=torch.int32, device=dev)
    cu = torch.tensor([0, tokens], dtype=torch.int32, device=dev)
    pos = torch.arange(context, context + tokens, dtype=torch.int32, device=dev)
    big, side = torch.zeros(1 << 28, device=dev), torch.cuda.Stream()

    def block(stream):
        cache = mx.kv4_cache(pages, H, D, page, dev)
        mx.kv4_append_into(old[:, :H], old[:, H:], torch.arange(context, device=dev), cache)
        torch.full((1 << 24,), 255, dtype=torch.uint8, device=dev)  # freed: fresh memory need not be zero
        torch.cuda.synchronize()
        for _ in range(10):
            big.add_(1)  # the current stream is busy
        b = AttentionBlock(w, qkv, o, Hq, cache, None, tokens, 1, tokens, pages)
        assert torch.cuda.current_stream().query()  # and the block ready for any other
        out = b.run(r, table, lens, cu, pos.long(), pos, stream=stream)
        torch.cuda.synchronize()
        mx.sync_status()
        assert not b.ws_att[:4096].any()
        return out

    assert torch.equal(block(side), block(None))
