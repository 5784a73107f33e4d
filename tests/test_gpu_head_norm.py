"""Norms of query and key heads with the rotation on the GPU.  GPU only."""
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


def _case(dev, T, Hq, H, D, seed=0):
    g = torch.Generator(device=dev).manual_seed(seed + T + Hq + D)
    qkv = (torch.randn((T, Hq + 2 * H, D), generator=g, device=dev) * 3).half()
    w = [(1 + 0.3 * torch.randn(D, generator=g, device=dev)).half() for _ in range(2)]
    pos = torch.randint(0, 500, (T,), generator=g, device=dev, dtype=torch.int32)
    return qkv, w, pos


def _tolerance(want, mag, D):
    """One rounding to fp16; before it, of the terms' magnitudes, the roundings of the weight times the table, the
    products, their sum and the norm's factor, which is off by half of its sum's (up to D / 16 + 8 roundings a sum in
    lanes and a tree) and its own few."""
    return 2.0 ** -11 * want.abs() + (D / 16 + 24) * 2.0 ** -24 * mag + 2.0 ** -25


@pytest.mark.parametrize("T,Hq,H,D", [(1, 32, 8, 128), (1, 1, 1, 64), (5, 7, 3, 64), (33, 4, 1, 256), (300, 6, 2, 128),
                                      (2100, 40, 8, 128), (4100, 9, 2, 64)])
@pytest.mark.parametrize("part", [0, 1, 2])
def test_against_the_formula(dev, T, Hq, H, D, part):
    rotary = (0, D // 2, D)[part]
    qkv, (w_q, w_k), pos = _case(dev, T, Hq, H, D)
    rope = mx.rope_table(512, rotary, device=dev) if rotary else None
    q, k, _ = qkv.split((Hq, H, H), 1)
    before = qkv.clone()
    out = torch.full((T, Hq + H + 1, D), 77.0, dtype=torch.float16, device=dev)  # rows apart
    mx.head_norm_rope_into(q, out[:, :Hq], w_q, k=k, k_out=out[:, Hq:Hq + H], w_k=w_k, positions=pos if rotary else None,
                           rope=rope, eps=1e-5)
    mx.sync_status()
    assert (out[:, -1] == 77).all() and torch.equal(qkv, before)
    for x, w, got in ((q, w_q, out[:, :Hq]), (k, w_k, out[:, Hq:Hq + H])):
        want, mag = ref.turned(x, w, 1e-5, rope, pos, rotary)
        off = (got.double() - want).abs()
        assert (off <= _tolerance(want, mag, D)).all()


@pytest.mark.parametrize("D", [64, 128])
def test_without_norms_it_is_the_rotation_alone(dev, D):
    qkv, _, pos = _case(dev, 50, 5, 2, D)
    rope = mx.rope_table(512, D // 2, device=dev)
    q, k, _ = qkv.split((5, 2, 2), 1)
    out = torch.empty((50, 7, D), dtype=torch.float16, device=dev)
    mx.head_norm_rope_into(q, out[:, :5], k=k, k_out=out[:, 5:], positions=pos, rope=rope)
    want = kv4_ref.rotate(qkv[:, :7].cpu().numpy(), rope.cpu().numpy(), pos.cpu().numpy(), D // 2)
    assert np.array_equal(out.cpu().numpy().view(np.uint16), want.view(np.uint16))


def test_one_side_only_and_in_place(dev):
    T, Hq, H, D = 20, 4, 2, 128
    qkv, (w_q, w_k), pos = _case(dev, T, Hq, H, D)
    rope = mx.rope_table(512, D, device=dev)
    q, k, _ = qkv.split((Hq, H, H), 1)
    want = torch.empty((T, Hq + H, D), dtype=torch.float16, device=dev)
    mx.head_norm_rope_into(q, want[:, :Hq], w_q, k=k, k_out=want[:, Hq:], w_k=None, positions=pos, rope=rope)
    only_q = torch.empty((T, Hq, D), dtype=torch.float16, device=dev)
    mx.head_norm_rope_into(q, only_q, w_q, positions=pos, rope=rope)
    mx.head_norm_rope_into(q, q, w_q, k=k, k_out=k, w_k=None, positions=pos, rope=rope)
    mx.sync_status()
    assert torch.equal(only_q, want[:, :Hq]) and torch.equal(qkv[:, :Hq + H], want)


def test_rows_of_zeros_and_of_what_is_not_finite(dev):
    D = 128
    x = torch.randn((4, 1, D), device=dev).half()
    x[0], x[1, 0, 5], x[2, 0, 7] = 0, float("nan"), float("inf")
    w, out = torch.ones(D, device=dev).half(), torch.empty_like(x)
    mx.head_norm_rope_into(x, out, w, eps=0.0)
    assert out[0].isnan().all()  # 0 times the reciprocal root of 0, by the formula
    mx.head_norm_rope_into(x, out, w)
    mx.sync_status()
    assert (out[0] == 0).all() and out[1].isnan().all() and out[3].isfinite().all()
    assert out[2, 0, 7].isnan() and (out[2, 0, :7] == 0).all()


def test_positions_that_are_skipped(dev):
    qkv, (w_q, w_k), pos = _case(dev, 6, 2, 1, 64)
    rope = mx.rope_table(512, 64, device=dev)
    want = torch.full((6, 2, 64), 77.0, dtype=torch.float16, device=dev)
    out = want.clone()
    mx.head_norm_rope_into(qkv[:, :2], want, w_q, positions=pos, rope=rope)
    pos[1] = pos[5] = -1
    mx.head_norm_rope_into(qkv[:, :2], out, w_q, positions=pos, rope=rope)
    mx.sync_status()  # padding is no error
    assert (out[[1, 5]] == 77).all() and torch.equal(out[[0, 2, 3, 4]], want[[0, 2, 3, 4]])
    pos[3] = 512
    out.fill_(77)
    mx.head_norm_rope_into(qkv[:, :2], out, w_q, positions=pos, rope=rope)
    with pytest.raises(_lib.MixLLMError) as e:
        mx.sync_status()
    assert e.value.status == _lib.ERR_BOUNDS
    assert (out[[1, 3, 5]] == 77).all() and torch.equal(out[[0, 2, 4]], want[[0, 2, 4]])


def test_bindings_check_their_tensors(dev):
    q = torch.ones((2, 3, 64), device=dev).half()
    w, i = torch.ones(64, device=dev).half(), torch.zeros(2, dtype=torch.int32, device=dev)
    rope = mx.rope_table(8, 64, device=dev)
    for bad in (lambda: mx.head_norm_rope_into(q, q, w[:32]), lambda: mx.head_norm_rope_into(q, q, w, k=q),
                lambda: mx.head_norm_rope_into(q, q, w, rope=rope), lambda: mx.head_norm_rope_into(q, q[:1], w),
                lambda: mx.head_norm_rope_into(q, q.float(), w), lambda: mx.head_norm_rope_into(q, q, w.float()),
                lambda: mx.head_norm_rope_into(q, q, w, positions=i[:1], rope=rope),
                lambda: mx.head_norm_rope_into(q.transpose(0, 1), q.transpose(0, 1), w),
                lambda: mx.head_norm_rope_into(q.cpu(), q.cpu(), w.cpu())):
        with pytest.raises(ValueError):
            bad()
    mx.head_norm_rope_into(q[:0], q[:0], w)
    mx.sync_status()
