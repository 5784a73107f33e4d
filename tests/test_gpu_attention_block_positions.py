"""layer.AttentionBlock skips a token whose position is out of range, with every
cache and with or without head norms: its slot is left as it was.  GPU only."""
import pytest

torch = pytest.importorskip("torch")

import mixed_precision_quantized_act_b200 as mx  # noqa: E402
from mixed_precision_quantized_act_b200 import _lib  # noqa: E402
from mixed_precision_quantized_act_b200.layer import AttentionBlock  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.load()
    return torch.device("cuda:0")


@pytest.mark.parametrize("wrong", [-1, 32, 2 ** 31 - 1])
@pytest.mark.parametrize("norms", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("cache_bits", [4, 8])
def test_a_position_out_of_range(dev, cache_bits, norms, wrong):
    Hq, H, D, page, K, B = 4, 2, 64, 16, 256, 3
    g = torch.Generator(device="cuda").manual_seed(3)
    randn = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    qkv, o = mx.w8a8_pack(randn((Hq + 2 * H) * D, K) * 0.05), mx.w8a8_pack(randn(K, Hq * D) * 0.05)
    w, w_q, w_k = torch.ones(K, device=dev).half(), (1 + 0.2 * randn(D)).half(), (1 + 0.2 * randn(D)).half()
    cache = (mx.kv8_cache if cache_bits == 8 else mx.kv4_cache)(8, H, D, page, dev)
    meta = cache.scales if cache_bits == 8 else cache.meta
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    table, cu = i32([[0], [1], [2]]), i32([0, 1, 2, 3])
    block = AttentionBlock(w, qkv, o, Hq, cache, mx.rope_table(32, D, device=dev), B, B, 1, 1,
                           w_q=w_q if norms[0] else None, w_k=w_k if norms[1] else None)
    slots = torch.arange(B, device=dev) * page
    block.run(randn(B, K).half(), table, i32([1, 1, 1]), cu, slots, i32([0, 0, 0]))  # leaves keys in every buffer
    mx.sync_status()
    q, codes, was = block.q.clone(), cache.codes.clone(), meta.clone()
    block.run(randn(B, K).half(), table, i32([2, 2, 2]), cu, slots + 1, i32([1, wrong, 1]))
    with pytest.raises(_lib.MixLLMError) as e:
        mx.sync_status()
    assert e.value.status == _lib.ERR_BOUNDS
    assert torch.equal(cache.codes[1], codes[1]) and torch.equal(meta[1], was[1]) and torch.equal(block.q[1], q[1])
    for b in (0, 2):
        assert not torch.equal(cache.codes[b], codes[b]) and not torch.equal(block.q[b], q[b])


def test_the_4_bit_append_checks_positions_without_a_table(dev):
    H, D, page, T = 2, 64, 16, 6
    kv = torch.randn((T, 2 * H, D), device=dev).half()
    slots, pos = torch.arange(T, device=dev), torch.arange(T, dtype=torch.int32, device=dev)
    k, v = kv.split((H, H), 1)
    want, cache = mx.kv4_cache(1, H, D, page, dev), mx.kv4_cache(1, H, D, page, dev)
    mx.kv4_append_into(k, v, slots, want)
    mx.kv4_append_into(k, v, slots, cache, positions=pos, max_pos=T)
    mx.sync_status()
    assert torch.equal(cache.codes, want.codes) and torch.equal(cache.meta, want.meta)
    cache = mx.kv4_cache(1, H, D, page, dev)
    pos[1], pos[4] = -1, T
    mx.kv4_append_into(k, v, slots, cache, positions=pos)  # nothing to check against
    mx.sync_status()
    assert torch.equal(cache.codes, want.codes)
    cache = mx.kv4_cache(1, H, D, page, dev)
    mx.kv4_append_into(k, v, slots, cache, positions=pos, max_pos=T)
    with pytest.raises(_lib.MixLLMError) as e:
        mx.sync_status()
    assert e.value.status == _lib.ERR_BOUNDS
    for t in range(T):
        row, held = cache.codes[0, :, :, t], want.codes[0, :, :, t]
        assert not row.any() and not cache.meta[0, :, :, t].any() if t in (1, 4) else torch.equal(row, held)
    with pytest.raises(ValueError):
        mx.kv4_append_into(k, v, slots, cache, max_pos=T)
    with pytest.raises(ValueError):
        mx.kv4_append_into(k, v, slots, cache, positions=pos[:2], max_pos=T)
