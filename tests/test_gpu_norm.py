"""The residual norms (mixllm_residual_norm) against their definition in 64
bits, and their codes against the quantizer's.  GPU only."""
import pytest

torch = pytest.importorskip("torch")

import mixed_precision_quantized_act_b200 as mx  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.load()
    return torch.device("cuda:0")


def _inputs(dev, M, K, kind, post, gate, seed=0):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x, r = rand(M, K).half(), (rand(M, K) * (1 + 19 * (torch.rand(K, generator=g) < 0.02))).to(kind)
    w = (1 + 0.2 * rand(K)).half()
    wp = (1 + 0.2 * rand(K)).half() if post else None
    gt = {"none": None, "channel": torch.sigmoid(rand(K)).half(), "row": torch.sigmoid(rand(1, K)).half(),
          "token": torch.sigmoid(rand(M, K)).half()}[gate]
    return [t if t is None else t.to(dev) for t in (x, r, w, wp, gt)]


def _reference(x, r, w, wp, gt, scale, eps, r_seen=None):
    """r' in 64 bits, and y from the rounded r' (the one given, or r)."""
    u = x.double()
    if wp is not None:
        u = u / (u.square().mean(-1, keepdim=True) + eps).sqrt() * wp.double()
    if gt is not None:
        u = u * gt.double()
    r2 = r.double() + scale * u
    seen = (r_seen if r_seen is not None else r2).double()
    return r2, scale * u, seen / (seen.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()


def _close(got, want, extra=0.0):
    """One rounding of got's type (half a step) plus fp32's own: a sum of K
    squares as a tree of at most 32 + 10 levels, rsqrt (2 ulp) and four products
    stay within 64 * 2^-24 of the terms in `extra`."""
    half_step = torch.finfo(got.dtype).eps / 2
    small = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps / 2
    off = (got.double() - want).abs()
    tol = half_step * want.abs() * (1 + 2.0 ** -10) + small + 64 * 2.0 ** -24 * (want.abs() + extra)
    return bool((off <= tol).all())


@pytest.mark.parametrize("M,K", [(1, 128), (3, 256), (1, 4096), (5, 8192), (130, 1152), (2, 14336), (2, 32768)])
@pytest.mark.parametrize("kind", [torch.float16, torch.float32])
@pytest.mark.parametrize("post,gate", [(False, "none"), (True, "channel"), (False, "token"), (True, "row")])
def test_norms_match_and_codes_are_the_quantizers(dev, M, K, kind, post, gate):
    x, r, w, wp, gt = _inputs(dev, M, K, kind, post, gate, seed=K)
    r_out, y = torch.empty_like(r), torch.empty_like(x)
    more = dict(x=x, r_out=r_out, w_post=wp, gate=gt, scale=0.75, eps=1e-5)
    mx.residual_norm_into(r, w, y, **more)
    mx.sync_status()
    r2, u, y2 = _reference(x, r, w, wp, gt, 0.75, 1e-5, r_out)
    assert _close(r_out, r2, u.abs() + r.double().abs())
    assert _close(y, y2)
    # the codes form: the same r', and the codes of y, bit for bit
    A_q, s_a = torch.empty((M, K), dtype=torch.int8, device=dev), torch.empty((M, K // 128), device=dev)
    r3, y3 = torch.empty_like(r), torch.empty_like(x)
    mx.residual_norm_quantize_into(r, w, A_q, s_a, y=y3, **{**more, "r_out": r3})
    A2, s2 = mx.quantize_act(y)
    assert torch.equal(r3, r_out) and torch.equal(y3, y) and torch.equal(A_q, A2) and torch.equal(s_a, s2)
    B_q, t_a = torch.empty_like(A_q), torch.empty_like(s_a)
    mx.residual_norm_quantize_into(r, w, B_q, t_a, **{**more, "r_out": None})
    assert torch.equal(B_q, A2) and torch.equal(t_a, s2)
    # and the way back
    back = mx.dequantize_act(A_q, s_a)
    assert torch.equal(back, (A_q.float() * s_a.repeat_interleave(128, 1)).half())
    mx.sync_status()


@pytest.mark.parametrize("kind", [torch.float16, torch.float32])
def test_in_place_strided_and_without_a_block(dev, kind):
    M, K = 37, 1280
    x, r, w, wp, gt = _inputs(dev, M, K, kind, True, "token")
    r_out, y = torch.empty_like(r), torch.empty_like(x)
    mx.residual_norm_into(r, w, y, x=x, r_out=r_out, w_post=wp, gate=gt)
    wide = torch.zeros((M, K + 64), dtype=kind, device=dev)
    wide[:, 16:16 + K] = r
    xs, gs = torch.zeros((M, 2 * K), dtype=torch.float16, device=dev), torch.zeros((M, K + 8), dtype=torch.float16, device=dev)
    xs[:, K:], gs[:, 8:] = x, gt
    inside, y2 = wide[:, 16:16 + K], torch.empty_like(y)
    mx.residual_norm_into(inside, w, y2, x=xs[:, K:], r_out=inside, w_post=wp, gate=gs[:, 8:])
    assert torch.equal(inside, r_out) and torch.equal(y2, y)
    assert not wide[:, :16].any() and not wide[:, 16 + K:].any()
    x2 = x.clone()
    mx.residual_norm_into(r, w, x2, x=x2, w_post=wp, gate=gt)  # y over x
    assert torch.equal(x2, y)
    keep = r.clone()
    mx.residual_norm_into(r, w, y)                             # no block: the norm before the first linear
    assert torch.equal(r, keep)
    assert _close(y, _reference(torch.zeros_like(x), r, w, None, None, 1.0, 1e-5)[2])
    mx.sync_status()


def test_zero_rows_and_values_that_are_not_finite(dev):
    M, K = 4, 256
    r, w = torch.zeros((M, K), device=dev), torch.ones(K, dtype=torch.float16, device=dev)
    r[1, 3], r[2, 7] = float("nan"), float("inf")
    r[3] = 1e-30
    y = torch.empty((M, K), dtype=torch.float16, device=dev)
    mx.residual_norm_into(r, w, y, eps=1e-6)
    assert (y[0] == 0).all() and y[1].isnan().all() and y[2, 7].isnan() and (y[2, :7] == 0).all() and (y[3] == 0).all()
    mx.residual_norm_into(r[:1], w, y[:1], eps=0.0)  # 0 * rsqrt(0): not a number, as the formula says
    assert y[0].isnan().all()


def test_empty_batches_and_refusals(dev):
    K = 256
    h = lambda *s: torch.zeros(s, dtype=torch.float16, device=dev)  # noqa: E731
    mx.residual_norm_into(h(0, K), h(K), h(0, K))
    mx.dequantize_act(torch.zeros((0, K), dtype=torch.int8, device=dev), torch.zeros((0, 2), device=dev))
    with pytest.raises(ValueError):
        mx.residual_norm_into(h(2, K), h(K + 8), h(2, K))
    with pytest.raises(ValueError):
        mx.residual_norm_into(h(2, K), h(K), h(2, K).float())
    with pytest.raises(ValueError):
        mx.residual_norm_into(h(2, K).cpu(), h(K), h(2, K))
    with pytest.raises(ValueError):
        mx.residual_norm_into(h(2, K), h(K), h(2, K), x=h(2, 2 * K)[:, ::2])
    with pytest.raises(mx.MixLLMError):
        mx.residual_norm_into(h(2, 200), h(200), h(2, 200))
    with pytest.raises(mx.MixLLMError):
        mx.residual_norm_into(h(2, K), h(K), h(2, K), r_out=h(2, K))        # r' without a block
    with pytest.raises(mx.MixLLMError):
        mx.residual_norm_into(h(2, K), h(K), h(2, K), x=h(2 * K + 8)[4:4 + 2 * K].view(2, K))  # 8-byte aligned
    mx.sync_status()
