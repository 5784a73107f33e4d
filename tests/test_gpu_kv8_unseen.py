"""Attention over the 8-bit cache where some query tokens of a request do not see
a block whose scale is NaN: only those that see it are lost.  GPU only."""
import pytest

torch = pytest.importorskip("torch")

import mixed_precision_quantized_act_b200 as mx  # noqa: E402
from tests import kv8_ref as ref  # noqa: E402
from tests.test_gpu_kv8 import _case, dev  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [2, 3, 4, 16, 40])
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("Hq,H,D", [(1, 1, 128), (4, 2, 64), (3, 1, 128), (4, 1, 64)])
def test_a_block_begun_by_a_later_query(dev, n, kind, Hq, H, D):  # noqa: F811
    """209 cached tokens, the last of which begins a block: the queries before it see nothing of that block, and their
    outputs and lse are those of a cache without it."""
    q, cache, table, lens, cu = _case(dev, [209], [n], Hq, H, D, 64, seed=n)
    scales = cache.scales.clone()
    scales[table[0, 3], kind, H - 1, 1] = float("nan")  # tokens 208 .. 223, keys or values of the last head
    out = torch.empty((n, Hq, D), dtype=torch.float16, device=dev)
    lse = torch.empty((n, Hq), device=dev)
    ws = mx.kv8_attention_workspace(1, n, Hq, cache, table.shape[1])
    mx.kv8_attention_into(q.to(dev), mx.KV8Cache(cache.codes, scales), table.to(dev), lens, cu, n, out, ws, lse=lse)
    mx.sync_status()
    lost = torch.zeros((n, Hq), dtype=torch.bool)
    lost[n - 1, Hq - Hq // H:] = True
    out, lse = out.cpu(), lse.cpu()
    assert out[lost].isnan().all()
    if kind == 0:  # a value's scale has no part in the score
        assert lse[lost].isnan().all()
    want, want_lse, tol = ref.attention(q, cache.codes.cpu(), cache.scales.cpu(), table, [209], cu.tolist(), D ** -0.5, True)
    assert ((out.double() - want).abs() <= tol)[~lost].all()
    # as for every lse: the relative errors of the probabilities' sum, and the rounding of the result
    far = (lse.double() - want_lse).abs()
    assert (far <= 2.0 ** -18 * (1 + want_lse.abs()) + 64 * D * 2.0 ** -24)[~lost].all()


@pytest.mark.parametrize("H,D", [(2, 128), (1, 64)])
def test_an_infinity_in_a_drafted_token(dev, H, D):  # noqa: F811
    """Three drafted tokens written behind 206 cached ones, the last with an infinity in its value, and checked at once:
    the first two are unharmed."""
    page, n = 64, 3
    _, cache, table, lens, cu = _case(dev, [209], [n], H, H, D, page, seed=1)
    g = torch.Generator(device=dev).manual_seed(5)
    kv = torch.randn((n, 2 * H, D), generator=g, device=dev).half()
    kv[2, H, 7] = float("inf")
    where = torch.arange(206, 209, device=dev)
    slots = table.to(dev)[0, where // page].long() * page + where % page
    mx.kv8_append_into(kv[:, :H], kv[:, H:], slots, cache)
    q = torch.randn((n, H, D), generator=g, device=dev).half()
    out = mx.kv8_attention(q, cache, table.to(dev), lens, cu, n).cpu()
    mx.sync_status()
    assert out[:2].isfinite().all() and out[2, 0].isnan().all() and out[2, 1:].isfinite().all()
    want, _, tol = ref.attention(q.cpu(), cache.codes.cpu(), cache.scales.cpu().nan_to_num(0.0), table, [209], cu.tolist(),
                                 D ** -0.5, True)
    assert ((out.double() - want).abs() <= tol)[:2].all()
