"""layer.AttentionBlock's checks that come before anything is allocated (CPU
only)."""
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

import mixed_precision_quantized_act_b200 as mx  # noqa: E402
from mixed_precision_quantized_act_b200.layer import AttentionBlock  # noqa: E402


def test_linears_on_another_device_are_refused():
    """A linear's kernels run on the cache's device: weights elsewhere are no
    addresses of its own."""
    cache = SimpleNamespace(kv_heads=2, head_dim=64, device=torch.device("cuda:0"))
    qkv, o = mx.empty_packed(512, 256, 0, "cpu"), mx.empty_packed(256, 256, 0, "cpu")
    with pytest.raises(ValueError, match="cache's device"):
        AttentionBlock(torch.ones(256, dtype=torch.float16), qkv, o, 4, cache, None, 1, 1, 1, 2)
