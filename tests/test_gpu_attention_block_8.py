"""layer.AttentionBlock with 8-bit linears, head norms and either cache: prompts
and then decode steps, each stage against its reference on the same inputs,
eagerly and as a replayed graph.  GPU only."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mixed_precision_quantized_act_b200 as mx  # noqa: E402
from mixed_precision_quantized_act_b200.layer import AttentionBlock  # noqa: E402
from tests import kv4_ref, kv8_ref  # noqa: E402
from tests.test_gpu_attention_block import _State  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.load()
    return torch.device("cuda:0")


def _linear(X, p):
    """The layer on these inputs, in 64 bits, and its tolerance: one rounding to fp16 and four of fp32."""
    q, s = kv8_ref.quantize_rows(X.cpu().numpy())
    y = torch.from_numpy(q).double() @ p.codes.cpu().double().t() * torch.from_numpy(s).double()[:, None] * p.s_w.cpu().double()
    return y, 2.0 ** -11 * y.abs() + 2.0 ** -21 * y.abs() + 2.0 ** -25


def _check(block, st, before, x, r, n, cache_before):
    r2 = before.double() + (x.double() if x is not None else 0)
    assert ((r.double() - r2).abs() <= 2.0 ** -11 * r2.abs() * 1.01 + 1e-7).all()
    want = r.double() / (r.double().square().mean(-1, keepdim=True) + block.eps).sqrt() * block.w_norm.double()
    assert ((block.y.double() - want).abs() <= 2.0 ** -11 * want.abs() * 1.01 + 2.0 ** -24).all()
    y, tol = _linear(block.y, block.qkv)
    heads = block.heads.view(block.tokens, -1).cpu().double()
    assert ((heads - y).abs() <= tol).all()
    Hq, H, D = block.q_heads, block.cache.kv_heads, block.cache.head_dim
    q, k, v = block.heads[:n].split((Hq, H, H), 1)
    got_q, got_k = torch.empty((n, Hq, D), device=r.device).half(), torch.empty((n, H, D), device=r.device).half()
    mx.head_norm_rope_into(q, got_q, block.w_q, k=k, k_out=got_k, w_k=block.w_k, positions=st.pos[:n].clone(),
                           rope=block.rope, eps=block.head_eps)
    assert torch.equal(block.q[:n], got_q)
    slots, page = st.slots[:n].cpu().numpy(), block.cache.page_size
    if block.eight:
        codes, scales = kv8_ref.append(*cache_before, slots.tolist(), got_k.cpu().numpy(), v.cpu().numpy())
        assert np.array_equal(block.cache.codes.cpu().numpy(), codes)
        assert np.array_equal(block.cache.scales.cpu().numpy(), scales)
        attention = kv8_ref.attention(block.q.cpu(), torch.from_numpy(codes), torch.from_numpy(scales), st.table.cpu(),
                                      st.lens.tolist(), st.cu.tolist(), D ** -0.5, True)
    else:
        codes, meta = block.cache.codes.cpu(), block.cache.meta.cpu()
        for kind, rows in ((0, got_k), (1, v)):
            by, m = kv4_ref.pack(*kv4_ref.quantize_row(rows.cpu().numpy()))
            at = (torch.from_numpy(slots // page), kind, slice(None), torch.from_numpy(slots % page))
            assert np.array_equal(codes[at].numpy(), by) and np.array_equal(meta[at].numpy().view(np.uint32), m)
        attention = kv4_ref.attention(block.q.cpu(), codes, meta, st.table.cpu(), st.lens.tolist(), st.cu.tolist(),
                                      D ** -0.5, True)
    want, _, tol = attention
    assert ((block.att[:n].cpu().double() - want[:n]).abs() <= tol[:n]).all()
    y, tol = _linear(block.att.view(block.tokens, -1), block.o_proj)
    assert ((block.out.cpu().double() - y).abs() <= tol).all()


@pytest.mark.parametrize("cache_bits", [4, 8])
@pytest.mark.parametrize("Hq,H,D,page", [(8, 2, 64, 16), (6, 3, 128, 64)])
def test_prompts_then_decode_steps(dev, cache_bits, Hq, H, D, page):
    K, B = 512, 3
    g = torch.Generator(device="cuda").manual_seed(7)
    randn = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    qkv, o = mx.w8a8_pack(randn((Hq + 2 * H) * D, K) * 0.04), mx.w8a8_pack(randn(K, Hq * D) * 0.04)
    w, w_q, w_k = (1 + 0.1 * randn(K)).half(), (1 + 0.2 * randn(D)).half(), (1 + 0.2 * randn(D)).half()
    cache = (mx.kv8_cache if cache_bits == 8 else mx.kv4_cache)(40, H, D, page, dev)
    rope, width = mx.rope_table(256, D, 10000.0, dev), -(-200 // page) + 1

    def held():
        return (cache.codes.cpu().numpy(), cache.scales.cpu().numpy()) if cache_bits == 8 else None

    # ---- prompts of different lengths, padded to 100 tokens
    st = _State(B, 40, width, 100, dev)
    st.new.copy_(torch.tensor([37, 0, 52], dtype=torch.int32))
    block = AttentionBlock(w, qkv, o, Hq, cache, rope, 100, B, 52, width, w_q=w_q, w_k=w_k)
    r = randn(100, K).half()
    before, was = r.clone(), held()
    st.assign(page)
    block.run(r, st.table, st.lens, st.cu, st.slots, st.pos)
    mx.sync_status()
    assert int(st.status) == 0
    _check(block, st, before, None, r, 89, was)

    # ---- decode steps over the same cache, eagerly once and then as a graph
    st.resize(B, dev)
    st.new.fill_(1)
    step = AttentionBlock(w, qkv, o, Hq, cache, rope, B, B, 1, width, w_q=w_q, w_k=w_k)
    r, x = torch.zeros((B, K), dtype=torch.float16, device=dev), torch.zeros((B, K), dtype=torch.float16, device=dev)

    def one():
        st.assign(page)
        step.run(r, st.table, st.lens, st.cu, st.slots, st.pos, x)

    def feed():
        r.copy_(randn(B, K))
        x.copy_(randn(B, K))
        return r.clone(), held()

    before, was = feed()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one()
    torch.cuda.current_stream().wait_stream(side)
    mx.sync_status()
    _check(step, st, before, x, r, B, was)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one()
    for _ in range(20):
        before, was = feed()
        graph.replay()
    mx.sync_status()
    assert int(st.status) == 0 and st.lens.tolist() == [58, 21, 73]
    _check(step, st, before, x, r, B, was)


def test_linears_of_both_kinds_in_one_block(dev):
    """A W4.4A8 qkv with an 8-bit o_proj and the other way round: each stage is the linear's own call."""
    Hq, H, D, page, K, B = 4, 2, 64, 16, 256, 2
    g = torch.Generator(device="cuda").manual_seed(3)
    randn = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    W_qkv, W_o, w = randn((Hq + 2 * H) * D, K) * 0.05, randn(K, Hq * D) * 0.05, torch.ones(K, device=dev).half()
    four = [mx.pack_weights(W, torch.zeros(W.shape[0], dtype=torch.uint8, device=dev)) for W in (W_qkv, W_o)]
    eight = [mx.w8a8_pack(W) for W in (W_qkv, W_o)]
    for qkv, o in ((four[0], eight[1]), (eight[0], four[1])):
        cache = mx.kv8_cache(8, H, D, page, dev)
        st = _State(B, 8, 4, B, dev)
        st.new.fill_(1)
        block = AttentionBlock(w, qkv, o, Hq, cache, None, B, B, 1, 4)
        r = randn(B, K).half()
        st.assign(page)
        block.run(r, st.table, st.lens, st.cu, st.slots, st.pos)
        mx.sync_status()
        y = torch.empty((B, K), dtype=torch.float16, device=dev)
        mx.residual_norm_into(r, w, y)
        heads = mx.w8a8_linear(y, qkv) if isinstance(qkv, mx.W8Weights) else mx.linear(y, qkv)
        assert torch.equal(block.heads.view(B, -1), heads)
        att = block.att.view(B, -1)
        out = mx.w8a8_linear(att, o) if isinstance(o, mx.W8Weights) else mx.linear(att, o)
        assert torch.equal(block.out, out)
