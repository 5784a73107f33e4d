"""Scores of keys whose sums cancel: one outlier channel decides a row's scale
and zero point, the other codes equal the zero point, and sum q code and
z sum q are far larger than their difference.  The logarithm of the softmax's
denominator is then the score itself (one token) or close to the largest one.
GPU only."""
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


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("z", [0, 15])
@pytest.mark.parametrize("kv", [1, 5])
@pytest.mark.parametrize("n,Hq,H", [(1, 4, 2), (3, 4, 1), (20, 4, 4)])  # one and two 8-row tiles, the prompt kernel
def test_scores_of_outlier_keys(dev, D, z, kv, n, Hq, H):
    B, page = 32, 16
    g = torch.Generator().manual_seed(D + z + kv + n)
    rand = lambda *s: torch.rand(s, generator=g)  # noqa: E731
    codes = torch.full((B, 2, H, page, D), z, dtype=torch.uint8)
    codes[:, 0].scatter_(3, torch.randint(0, D, (B, H, page, 1), generator=g), 15 - z)
    codes[:, 1] = torch.randint(0, 16, codes[:, 1].shape, generator=g, dtype=torch.uint8)
    by = codes[..., 0::2] | codes[..., 1::2] << 4
    s = (rand(B, 2, H, page) * 3 + 1).half()
    meta = (s.view(torch.int16).to(torch.int32) & 0xFFFF) | z << 16
    cache = mx.KV4Cache(by.to(dev), meta.to(dev))
    q = torch.randn((B * n, Hq, D), generator=g) * (1 + 9 * (rand(D) < 0.1))
    q = q.half().to(dev)
    table = torch.arange(B, dtype=torch.int32, device=dev)[:, None]
    lens = torch.full((B,), kv, dtype=torch.int32, device=dev)
    cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device=dev)
    out, lse = torch.empty_like(q), torch.empty((B * n, Hq), device=dev)
    ws = mx.kv4_attention_workspace(B, n, Hq, cache, 1)
    mx.kv4_attention_into(q, cache, table, lens, cu, n, out, ws, causal=False, lse=lse)
    mx.sync_status()
    want, want_lse, tol, lse_tol = kv4_exact.attention(q, cache, table, lens, cu, D ** -0.5, False)
    off = kv4_exact.off_by(out, want, tol), kv4_exact.off_by(lse, want_lse, lse_tol)
    assert max(off) <= 1, off
    # what the header promises of a score, and the rounding of the logarithm itself
    x = q.double().abs()
    bound = 4 * D ** -0.5 * (D * 2.0 ** -18 * x.amax(-1) + (D + 16) * 2.0 ** -19 * x.sum(-1))
    far = (lse.double() - want_lse).abs()
    assert (far <= bound + 2.0 ** -20 + 2.0 ** -22 * (want_lse.abs() + 200)).all()

