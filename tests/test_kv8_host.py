"""The 8-bit operators' entry points reject bad arguments on the host, before any
device call, and size their workspaces there (CPU only)."""
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
    return list({**args, **by}.values())


PACK = dict(W=P(0x1000), N=3, K=64, codes=P(0x2000), s=P(0x3000), stream=None)


@pytest.mark.parametrize("by,status", [
    (dict(K=0), UNSUPPORTED), (dict(K=-16), UNSUPPORTED), (dict(K=72), UNSUPPORTED), (dict(K=131072), UNSUPPORTED),
    (dict(N=-1), BAD), (dict(N=2 ** 31), BAD), (dict(W=None), BAD), (dict(codes=None), BAD), (dict(s=None), BAD),
    (dict(W=P(0x1008)), BAD), (dict(codes=P(0x2008)), BAD), (dict(s=P(0x3002)), BAD), (dict(N=0, W=None), OK)])
def test_pack(L, by, status):
    assert L.mixllm_w8a8_pack(*_changed(PACK, **by)) == status


QUANT = dict(X=P(0x1000), stride=64, M=3, K=64, A=P(0x2000), s=P(0x3000), stream=None)


@pytest.mark.parametrize("by,status", [
    (dict(K=40), UNSUPPORTED), (dict(M=-1), BAD), (dict(X=None), BAD), (dict(A=None), BAD), (dict(s=None), BAD),
    (dict(X=P(0x1002)), BAD), (dict(stride=65), BAD), (dict(A=P(0x2004)), BAD), (dict(M=0, X=None), OK)])
def test_quantize(L, by, status):
    assert L.mixllm_w8a8_quantize(*_changed(QUANT, **by)) == status


GEMM = dict(A=P(0x1000), s_a=P(0x2000), M=3, K=64, W=P(0x3000), s_w=P(0x4000), N=5, bias=None, Y=P(0x5000), stream=None)
LINEAR = dict(X=P(0x1000), stride=64, M=3, K=64, W=P(0x3000), s_w=P(0x4000), N=5, bias=None, Y=P(0x5000), ws=P(0x6000),
              ws_bytes=1 << 20, stream=None)
BOTH = [(dict(K=24), UNSUPPORTED), (dict(K=131072), UNSUPPORTED), (dict(M=-1), BAD), (dict(N=-1), BAD), (dict(M=2 ** 31), BAD),
        (dict(W=None), BAD), (dict(s_w=None), BAD), (dict(Y=None), BAD), (dict(W=P(0x3008)), BAD), (dict(s_w=P(0x4002)), BAD),
        (dict(bias=P(0x7001)), BAD), (dict(Y=P(0x5001)), BAD), (dict(M=0, W=None), OK), (dict(N=0, Y=None), OK)]


@pytest.mark.parametrize("by,status", BOTH + [(dict(A=None), BAD), (dict(s_a=None), BAD), (dict(A=P(0x1004)), BAD),
                                              (dict(s_a=P(0x2002)), BAD)])
def test_gemm(L, by, status):
    assert L.mixllm_w8a8_gemm(*_changed(GEMM, **by)) == status


@pytest.mark.parametrize("by,status", BOTH + [(dict(X=None), BAD), (dict(X=P(0x1008)), BAD), (dict(stride=60), BAD),
                                              (dict(ws=None), BAD), (dict(ws=P(0x6010)), BAD), (dict(ws_bytes=511), BAD)])
def test_linear(L, by, status):
    assert L.mixllm_w8a8_linear(*_changed(LINEAR, **by)) == status


def test_linear_workspace(L):
    def ws(M, K, N):
        out = ctypes.c_size_t(77)
        return L.mixllm_w8a8_linear_workspace_bytes(M, K, N, ctypes.byref(out)), out.value

    assert ws(3, 64, 5) == (OK, 256 + 256)  # codes, then scales
    assert ws(1000, 4096, 7) == (OK, 1000 * 4096 + 4096)
    assert ws(0, 64, 5) == (OK, 0) and ws(3, 64, 0) == (OK, 0)
    assert ws(3, 8, 5)[0] == UNSUPPORTED and ws(-1, 64, 5)[0] == BAD
    assert L.mixllm_w8a8_linear_workspace_bytes(1, 64, 5, None) == BAD


HEADS = dict(q=P(0x100), qs=512, Hq=4, qo=P(0x200), qos=512, wq=P(0x300), k=P(0x400), ks=256, H=2, ko=P(0x500), kos=256,
             wk=P(0x600), T=3, D=128, eps=1e-6, pos=P(0x700), rope=P(0x800), max_pos=9, rotary=128, stream=None)


@pytest.mark.parametrize("by,status", [
    (dict(D=96), UNSUPPORTED), (dict(D=512), UNSUPPORTED), (dict(rotary=24), UNSUPPORTED), (dict(rotary=144), UNSUPPORTED),
    (dict(rotary=-16), UNSUPPORTED), (dict(T=-1), BAD), (dict(Hq=-1), BAD), (dict(H=-1), BAD), (dict(eps=-1.0), BAD),
    (dict(eps=float("nan")), BAD), (dict(q=None), BAD), (dict(qo=None), BAD), (dict(k=None), BAD), (dict(ko=None), BAD),
    (dict(rope=None), BAD), (dict(pos=None), BAD), (dict(max_pos=0), BAD), (dict(q=P(0x108)), BAD), (dict(wq=P(0x302)), BAD),
    (dict(wk=P(0x604)), BAD), (dict(rope=P(0x804)), BAD), (dict(qs=4), BAD), (dict(qos=504), BAD), (dict(kos=248), BAD),
    (dict(T=0, q=None), OK), (dict(Hq=0, H=0, q=None), OK)])
def test_head_norm_rope(L, by, status):
    assert L.mixllm_head_norm_rope(*_changed(HEADS, **by)) == status


CACHE = dict(codes=P(0x1000), scales=P(0x2000), pages=4, H=2, D=128, page=64)
BAD_CACHES = [(dict(page=24), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED),
              (dict(H=0), BAD), (dict(pages=-1), BAD), (dict(codes=None), BAD), (dict(scales=P(0x2008)), BAD)]
APPEND = dict(CACHE, slots=P(0x10), n=3, k=P(0x20), ks=256, v=P(0x30), vs=256, q=P(0x40), qs=512, Hq=4, qo=P(0x50),
              qos=512, wq=P(0x60), wk=P(0x70), eps=1e-6, pos=P(0x80), rope=P(0x90), max_pos=100, rotary=128, stream=None)


@pytest.mark.parametrize("by,status", BAD_CACHES + [
    (dict(n=-1), BAD), (dict(n=0, slots=None, k=None), OK), (dict(slots=None), BAD), (dict(slots=P(0x14)), BAD),
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(q=None), BAD), (dict(qo=None), BAD), (dict(Hq=-1), BAD),
    (dict(rotary=24), UNSUPPORTED), (dict(rotary=144), UNSUPPORTED), (dict(rope=None), BAD), (dict(pos=None), BAD),
    (dict(max_pos=0), BAD), (dict(k=P(0x28)), BAD), (dict(ks=257), BAD), (dict(vs=4), BAD), (dict(qs=4), BAD),
    (dict(qos=504), BAD), (dict(wq=P(0x62)), BAD), (dict(eps=-1.0), BAD)])
def test_append(L, by, status):
    assert L.mixllm_kv8_append(*_changed(APPEND, **by)) == status


READ = dict(CACHE, slots=P(0x10), n=3, k=P(0x20), v=P(0x30), stream=None)


@pytest.mark.parametrize("by,status", BAD_CACHES + [(dict(n=-1), BAD), (dict(n=0, k=None), OK), (dict(k=None), BAD),
                                                    (dict(v=P(0x38)), BAD), (dict(slots=None), BAD)])
def test_read(L, by, status):
    assert L.mixllm_kv8_read(*_changed(READ, **by)) == status


ATTEND = dict(q=P(0x100), qs=512, T=3, Hq=4, codes=P(0x1000), scales=P(0x2000), pages=4, H=2, D=128, page=64,
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
    assert L.mixllm_kv8_attention(*_changed(ATTEND, **by)) == status


def test_attention_workspace(L):
    def ws(B=2, max_q=1, Hq=8, H=2, D=128, page=64, W=8):
        out = ctypes.c_size_t(0)
        return L.mixllm_kv8_attention_workspace_bytes(B, max_q, Hq, H, D, page, W, ctypes.byref(out)), out.value

    # up to 16 rows a request: counters and the parts of 148 blocks (two each, and one per warp), whatever the batch
    for B in (1, 2, 16384):
        assert ws(B) == (OK, 4096 + 148 * 10 * 8 * (128 + 12) * 4)
    assert ws(max_q=4) == (OK, 4096 + 148 * 10 * 16 * (128 + 12) * 4)
    # more rows: the 4-bit cache's
    for B, max_q in ((1, 5), (3, 1000)):
        pairs = B * -(-max_q * 4 // 256)
        plan = (4096 + 8 * (pairs + 1) + 8 * pairs + 255) // 256 * 256
        assert ws(B, max_q) == (OK, 4096 + plan + 148 * 2 * 256 * (128 + 2) * 4)
    assert ws(D=80)[0] == UNSUPPORTED and ws(Hq=7)[0] == BAD and ws(B=16385)[0] == UNSUPPORTED
    assert L.mixllm_kv8_attention_workspace_bytes(1, 1, 8, 2, 128, 64, 8, None) == BAD


def test_bindings_reject_host_tensors(L):
    torch = pytest.importorskip("torch")
    import mixed_precision_quantized_act_b200 as mx
    z = lambda *s, dtype=torch.float16: torch.zeros(s, dtype=dtype)  # noqa: E731
    for bad in (lambda: mx.kv8_cache(2, 1, 64, 16, "cpu"), lambda: mx.w8a8_pack(z(2, 64, dtype=torch.float32)),
                lambda: mx.W8Weights(z(2, 64, dtype=torch.int8), z(2, dtype=torch.float32)),
                lambda: mx.w8a8_quantize(z(2, 64)), lambda: mx.head_norm_rope_into(z(2, 1, 64), z(2, 1, 64))):
        with pytest.raises(ValueError):
            bad()
