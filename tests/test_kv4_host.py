"""The KV-cache and norm entry points reject bad arguments on the host, before
any device call, and size their workspaces there (CPU only)."""
import ctypes

import pytest

from mixed_precision_quantized_act_b200 import _lib
from mixed_precision_quantized_act_b200 import build as libbuild

P = ctypes.c_void_p
BAD, UNSUPPORTED, OK = _lib.ERR_INVALID_ARG, _lib.ERR_UNSUPPORTED, _lib.OK


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return _lib.load()


def _changed(args, **by):
    out = dict(args)
    out.update(by)
    return list(out.values())


NORM = dict(r=P(0x1000), r_stride=256, f32=0, x=P(0x2000), x_stride=256, w_post=P(0x3000), gate=P(0x4000),
            gate_stride=256, scale=1.0, r_out=P(0x5000), r_out_stride=256, w=P(0x6000), eps=1e-5, M=2, K=256,
            y=P(0x7000), A_q=P(0x8000), s_a=P(0x9000), stream=None)


@pytest.mark.parametrize("by,status", [
    (dict(K=200), UNSUPPORTED), (dict(K=0), UNSUPPORTED), (dict(K=32768 + 128), UNSUPPORTED), (dict(M=-1), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(r=None), BAD), (dict(w=None), BAD),
    (dict(y=None, A_q=None, s_a=None), BAD), (dict(s_a=None), BAD), (dict(A_q=None), BAD), (dict(x=None), BAD),
    (dict(x=None, w_post=None, gate=None), BAD), (dict(r=P(0x1008)), BAD), (dict(A_q=P(0x8004)), BAD),
    (dict(r_stride=252), BAD), (dict(r_stride=252, f32=1, r_out_stride=254), BAD), (dict(x_stride=257), BAD),
    (dict(gate_stride=4), BAD), (dict(r_out_stride=128), BAD), (dict(M=0, r=None), OK)])
def test_residual_norm(L, by, status):
    assert L.mixllm_residual_norm(*_changed(NORM, **by)) == status


def test_dequantize_act(L):
    f = L.mixllm_dequantize_act
    assert f(P(8), P(8), 1, 200, 128, P(16), None) == UNSUPPORTED
    assert f(P(8), P(8), 1, 256, 64, P(16), None) == UNSUPPORTED
    assert f(P(8), P(8), -1, 256, 128, P(16), None) == BAD
    assert f(None, P(8), 1, 256, 128, P(16), None) == BAD
    assert f(P(8), P(8), 1, 256, 128, P(24), None) == BAD
    assert f(None, None, 0, 256, 128, None, None) == OK


ASSIGN = dict(ctx=P(0x10), new=P(0x20), B=4, table=P(0x30), stride=8, width=8, free=P(0x40), n_free=9, count=P(0x50),
              page=64, seq=P(0x60), cu=P(0x70), slots=P(0x80), pos=P(0x90), T=5, left=P(0xA0), status=P(0xB0),
              stream=None)


@pytest.mark.parametrize("by,status", [
    (dict(page=48), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=512), UNSUPPORTED), (dict(B=-1), BAD),
    (dict(B=16385), UNSUPPORTED), (dict(width=-1), BAD), (dict(T=-1), BAD), (dict(n_free=-1), BAD),
    (dict(T=2 ** 31), BAD), (dict(width=2 ** 26), BAD), (dict(stride=7), BAD), (dict(ctx=None), BAD),
    (dict(table=None), BAD), (dict(free=None), BAD), (dict(count=None), BAD), (dict(cu=None), BAD),
    (dict(slots=None), BAD), (dict(status=None), BAD), (dict(left=None), BAD), (dict(slots=P(0x84)), BAD),
    (dict(ctx=P(0x11)), BAD)])
def test_assign(L, by, status):
    assert L.mixllm_kv4_assign(*_changed(ASSIGN, **by)) == status


CACHE = dict(codes=P(0x1000), meta=P(0x2000), pages=4, H=2, D=128, page=64)
APPEND = dict(CACHE, slots=P(0x10), n=3, k=P(0x20), ks=256, v=P(0x30), vs=256, q=P(0x40), qs=512, Hq=4, qo=P(0x50),
              qos=512, pos=P(0x60), rope=P(0x70), max_pos=100, rotary=128, stream=None)
BAD_CACHES = [(dict(page=24), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED), (dict(H=0), BAD),
              (dict(pages=-1), BAD), (dict(codes=None), BAD), (dict(meta=P(0x2008)), BAD)]


@pytest.mark.parametrize("by,status", BAD_CACHES + [
    (dict(n=-1), BAD), (dict(n=0, slots=None, k=None), OK), (dict(slots=None), BAD), (dict(k=None), BAD),
    (dict(q=None), BAD), (dict(qo=None), BAD), (dict(Hq=-1), BAD), (dict(rotary=24), UNSUPPORTED),
    (dict(rotary=144), UNSUPPORTED), (dict(rotary=-16), UNSUPPORTED), (dict(rope=None), BAD), (dict(pos=None), BAD),
    (dict(max_pos=0), BAD), (dict(k=P(0x28)), BAD), (dict(ks=257), BAD), (dict(qs=4), BAD), (dict(qos=504), BAD),
    (dict(slots=P(0x14)), BAD)])
def test_append(L, by, status):
    assert L.mixllm_kv4_append(*_changed(APPEND, **by)) == status


READ = dict(CACHE, slots=P(0x10), n=3, k=P(0x20), v=P(0x30), stream=None)


@pytest.mark.parametrize("by,status", BAD_CACHES + [(dict(n=-1), BAD), (dict(n=0, k=None), OK), (dict(k=None), BAD),
                                                    (dict(v=P(0x38)), BAD), (dict(slots=None), BAD)])
def test_read(L, by, status):
    assert L.mixllm_kv4_read(*_changed(READ, **by)) == status


ATTEND = dict(q=P(0x100), qs=512, T=3, Hq=4, codes=P(0x1000), meta=P(0x2000), pages=4, H=2, D=128, page=64,
              table=P(0x200), ts=8, W=8, lens=P(0x300), cu=P(0x400), B=2, max_q=2, scale=0.1, causal=1, out=P(0x500),
              os=512, lse=None, ws=P(0x10000), ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("by,status", BAD_CACHES + [
    (dict(Hq=3), BAD), (dict(Hq=1), BAD), (dict(B=-1), BAD), (dict(B=16385), UNSUPPORTED), (dict(max_q=-1), BAD),
    (dict(max_q=2 ** 31), BAD), (dict(W=-1), BAD), (dict(W=2 ** 26), BAD), (dict(T=-1), BAD),
    (dict(scale=float("inf")), BAD), (dict(scale=float("nan")), BAD), (dict(q=None), BAD), (dict(out=None), BAD),
    (dict(lens=None), BAD), (dict(cu=None), BAD), (dict(table=None), BAD), (dict(q=P(0x108)), BAD),
    (dict(out=P(0x502)), BAD), (dict(qs=508), BAD), (dict(os=256), BAD), (dict(lse=P(0x602)), BAD),
    (dict(ws_bytes=100), BAD), (dict(ws=None), BAD), (dict(ws=P(0x10010)), BAD), (dict(T=0, q=None), OK),
    (dict(B=0), OK), (dict(max_q=0), OK)])
def test_attention(L, by, status):
    assert L.mixllm_kv4_attention(*_changed(ATTEND, **by)) == status


def test_attention_workspace(L):
    def ws(B=2, max_q=1, Hq=8, H=2, D=128, page=64, W=8):
        out = ctypes.c_size_t(0)
        return L.mixllm_kv4_attention_workspace_bytes(B, max_q, Hq, H, D, page, W, ctypes.byref(out)), out.value

    # up to 16 rows (queries x heads of a group) a request: counters and the parts of 148 blocks (two each, and one
    # per warp), whatever the batch
    for B in (1, 2, 16384):
        assert ws(B) == (OK, 4096 + 148 * 18 * 8 * (128 + 12) * 4)
    assert ws(max_q=4) == (OK, 4096 + 148 * 18 * 16 * (128 + 12) * 4)
    assert ws(max_q=2, D=64) == (OK, 4096 + 148 * 18 * 8 * (64 + 12) * 4)
    # more rows: counters, the list of 256-row tile pairs, and two parts of 256 rows per block
    for B, max_q in ((1, 5), (3, 1000)):
        pairs = B * -(-max_q * 4 // 256)
        plan = (4096 + 8 * (pairs + 1) + 8 * pairs + 255) // 256 * 256
        assert ws(B, max_q) == (OK, 4096 + plan + 148 * 2 * 256 * (128 + 2) * 4)
    assert ws(D=80)[0] == UNSUPPORTED and ws(Hq=7)[0] == BAD and ws(B=16385)[0] == UNSUPPORTED
    assert L.mixllm_kv4_attention_workspace_bytes(1, 1, 8, 2, 128, 64, 8, None) == BAD


def test_bindings_reject_host_tensors(L):
    torch = pytest.importorskip("torch")
    import mixed_precision_quantized_act_b200 as mx
    z = lambda *s, dtype=torch.float16: torch.zeros(s, dtype=dtype)  # noqa: E731
    with pytest.raises(ValueError):
        mx.kv4_cache(2, 1, 64, 16, "cpu")
    with pytest.raises(ValueError):
        mx.residual_norm_into(z(2, 256), z(256), z(2, 256))
    with pytest.raises(ValueError):
        mx.dequantize_act(z(2, 256, dtype=torch.int8), z(2, 2, dtype=torch.float32))
    i = z(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        mx.kv4_assign_into(i, i, z(2, 3, dtype=torch.int32), i, i[:1], 16, i, i, z(4, dtype=torch.int64), i, i[:1], i[:1])


def test_rope_table_is_the_formula(L):
    torch = pytest.importorskip("torch")
    import math

    import mixed_precision_quantized_act_b200 as mx
    t = mx.rope_table(1000, 64, 500000.0, "cpu")
    assert t.shape == (1000, 64) and t.dtype is torch.float32
    for pos, i in ((0, 0), (999, 0), (999, 31), (123, 7)):
        angle = pos * 500000.0 ** (-2 * i / 64)
        assert abs(float(t[pos, i]) - math.cos(angle)) <= 2.0 ** -24
        assert abs(float(t[pos, 32 + i]) - math.sin(angle)) <= 2.0 ** -24
