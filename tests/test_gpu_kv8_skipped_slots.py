"""Lists of slots with skipped tokens inside a block: the append writes the block
as one, and records what lies too far behind its first token.  GPU only."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mixed_precision_quantized_act_b200 as mx  # noqa: E402
from mixed_precision_quantized_act_b200 import _lib  # noqa: E402
from tests import kv8_ref as ref  # noqa: E402
from tests.test_gpu_kv8 import _filled, dev  # noqa: E402,F401
from tests.test_kv8_runs_model import BLOCK, _header  # noqa: E402

pytestmark = pytest.mark.gpu


def _case(dev, slots, H, D, page, seed, scale, rope=False):  # noqa: F811
    """Appends to these slots; the cache against the definition on the places that the header names, bit for bit."""
    slots = list(slots)
    T, pages = len(slots), max(slots) // page + 2
    g = torch.Generator(device=dev).manual_seed(seed)
    cache = _filled(dev, pages, H, D, page, seed)
    codes, scales = cache.codes.cpu().numpy(), cache.scales.cpu().numpy()
    kv = (torch.randn((T, 3 * H, D), generator=g, device=dev) * scale).half()
    q, k, v = kv.split((H, H, H), 1)
    q_out, w = torch.full_like(q, 77.0).contiguous(), (1 + 0.2 * torch.randn(D, generator=g, device=dev)).half()
    turn = dict(positions=torch.arange(T, dtype=torch.int32, device=dev), rope=mx.rope_table(T, D, device=dev)) if rope else {}
    mx.kv8_append_into(k, v, torch.tensor(slots, device=dev), cache, q=q, q_out=q_out, w_q=w, w_k=w, **turn)
    runs, recorded = _header(slots)
    if recorded:
        with pytest.raises(_lib.MixLLMError) as e:
            mx.sync_status()
        assert e.value.status == _lib.ERR_BOUNDS
    else:
        mx.sync_status()
    want_q, want_k = torch.empty_like(q_out), torch.empty_like(q_out)
    mx.head_norm_rope_into(q, want_q, w, k=k, k_out=want_k, w_k=w, **turn)
    mx.sync_status()
    kept = {t for r in runs for t in r}
    codes, scales = ref.append(codes, scales, [s if t in kept else -1 for t, s in enumerate(slots)],
                               want_k.cpu().numpy(), v.cpu().numpy())
    assert np.array_equal(cache.scales.cpu().numpy(), scales) and np.array_equal(cache.codes.cpu().numpy(), codes)
    there = torch.tensor(slots, device=dev) >= 0  # queries go by their slot alone
    assert torch.equal(q_out[there], want_q[there]) and (q_out[~there] == 77).all()


LISTS = {
    "one": [0, 1, -1, 2], "first": [-1, 0, -1, -1, 1, 16, -1, 17], "edge": [14, 15, -1, 16],
    "last place": [0] + 14 * [-1] + [1], "two tiles": 10 * [-1] + [3, -1, 4] + 7 * [-1] + [5, 6],
    "every third left out": [t if t % 3 else -1 for t in range(7, 120)],
    "padding between": [5, 6] + 500 * [-1] + [32] + 130 * [-1] + [50, 51] + 33 * [-1] + [64, -1, 66] + 90 * [-1],
    "many": [s for r in range(60) for s in [r * 32 + t if (t * 7 + r) % 4 else -1 for t in range(r % 16, 20)] + (r % 5) * [-1]],
}
FAR = {
    "one behind": [0, 17] + 15 * [-1] + [18], "next tile": [3] + 15 * [-1] + [4, 5], "far": [0] + 40 * [-1] + [1, 32, 33],
    "very far": [1] + 700 * [-1] + [2, 3] + 90 * [-1] + [4], "a chain": [0] + 12 * [-1] + [1] + 12 * [-1] + [2, 3],
}


@pytest.mark.parametrize("name", LISTS)
@pytest.mark.parametrize("H,D,page", [(2, 128, 16), (3, 64, 64)])
def test_skipped_tokens_inside_a_block(dev, name, H, D, page):  # noqa: F811
    for scale in (3.0, 0.05):  # blocks that grow, and that do not
        _case(dev, LISTS[name], H, D, page, len(name), scale, rope=scale == 3.0)


@pytest.mark.parametrize("name", FAR)
@pytest.mark.parametrize("H,D,page", [(2, 128, 16), (1, 64, 64)])
def test_tokens_too_far_behind_are_recorded(dev, name, H, D, page):  # noqa: F811
    _case(dev, FAR[name], H, D, page, len(name), 2.0)


def test_lists_at_random(dev):  # noqa: F811
    """Requests in blocks of their own, tokens left out in their places: nothing is recorded, up to two kernels."""
    rng = np.random.default_rng(4)
    for most in (3, 30, 60):
        slots, block = [], 0
        for _ in range(most):
            first, n = int(rng.integers(BLOCK)), int(rng.choice([1, 2, 20, 45]))
            part = [block * BLOCK + t for t in range(first, first + n)]
            slots += [s if rng.random() < 0.7 else -1 for s in part] + [-1] * int(rng.choice([0, 3, 40]))
            block += -(-(first + n) // BLOCK)
        assert not _header(slots)[1] and max(slots) >= 0
        _case(dev, slots, 2, 128, 32, most, 3.0)
