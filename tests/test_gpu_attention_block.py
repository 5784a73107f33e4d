"""layer.AttentionBlock: prompts and then decode steps through page assignment,
norm, qkv linear, cache write, attention and o_proj, each stage against its
reference on the same inputs, eagerly and as a replayed graph.  GPU only."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
import mixed_precision_quantized_act_b200 as mx  # noqa: E402
from mixed_precision_quantized_act_b200 import workloads as wl  # noqa: E402
from mixed_precision_quantized_act_b200.layer import AttentionBlock  # noqa: E402
from tests import kv4_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.load()
    return torch.device("cuda:0")


def _packed(layer, dev):
    W, is8 = wl.make_w(layer, 3), wl.make_bitmap(layer, 3)
    return mx.pack_weights(torch.from_numpy(W).to(dev), torch.from_numpy(is8).to(dev)), oracle.Quantized(W, is8)


class _State:
    """Requests, pages and slots of a step, as device tensors."""

    def __init__(self, B, pages, width, tokens, dev):
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
        self.lens, self.new, self.status = i32([0] * B), i32([0] * B), i32([0])
        self.table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
        self.free, self.count = torch.randperm(pages, device=dev).to(torch.int32), i32([pages])
        self.cu = i32([0] * (B + 1))
        self.resize(tokens, dev)

    def resize(self, tokens, dev):
        self.slots = torch.full((tokens,), -1, dtype=torch.int64, device=dev)
        self.pos = torch.full((tokens,), -1, dtype=torch.int32, device=dev)

    def assign(self, page):
        mx.kv4_assign_into(self.lens, self.new, self.table, self.free, self.count, page, self.lens, self.cu, self.slots,
                           self.pos, self.count, self.status)


def _close(Y, Y_ref):
    """The linears' tolerance against the CPU oracle."""
    Y_ref = Y_ref.astype(np.float64)
    off = np.abs(Y.cpu().numpy().astype(np.float64) - Y_ref)
    return (off <= 2.0 ** -9 * np.abs(Y_ref) + 1e-3 * np.sqrt(np.mean(Y_ref ** 2))).all()


def _check_stages(block, st, r_before, x, r, w, oq, oo, n, scale):
    """Every stage of the pass just run, on the inputs that it saw.  n tokens are not padding."""
    r2 = r_before.double() + (x.double() if x is not None else 0)
    # one rounding of the residual's type, and the fused multiply-add's
    eps = torch.finfo(r.dtype).eps / 2
    assert ((r.double() - r2).abs() <= eps * r2.abs() * 1.01 + 1e-7).all()
    y = torch.empty((r.shape[0], r.shape[1]), dtype=torch.float16, device=r.device)
    mx.residual_norm_into(r, w, y, eps=block.eps)
    want = r.double() / (r.double().square().mean(-1, keepdim=True) + block.eps).sqrt() * w.double()
    assert ((y.double() - want).abs() <= 2.0 ** -11 * want.abs() * 1.01 + 2.0 ** -24).all()
    A_o, s_o = oracle.quantize_act(y.cpu().numpy())
    assert np.array_equal(block.A_q.cpu().numpy(), A_o) and np.array_equal(block.s_a.cpu().numpy(), s_o)
    assert _close(block.heads.view(block.tokens, -1), oracle.gemm_w4w8a8(A_o, s_o, oq))
    Hq, H = block.q_heads, block.cache.kv_heads
    heads = block.heads.cpu().numpy()
    pos = st.pos[:n].cpu().numpy()
    rot = ref.rotate(heads[:n, :Hq + H], block.rope.cpu().numpy(), pos, block.rope.shape[1])
    assert np.array_equal(block.q[:n].cpu().numpy().view(np.uint16), rot[:, :Hq].view(np.uint16))
    slots, page = st.slots[:n].cpu().numpy(), block.cache.page_size
    codes, meta = block.cache.codes.cpu(), block.cache.meta.cpu()
    for kind, rows in ((0, rot[:, Hq:]), (1, heads[:n, Hq + H:])):
        by, m = ref.pack(*ref.quantize_row(rows))
        at = (torch.from_numpy(slots // page), kind, slice(None), torch.from_numpy(slots % page))
        assert np.array_equal(codes[at].numpy(), by) and np.array_equal(meta[at].numpy().view(np.uint32), m)
    want, _, tol = ref.attention(block.q.cpu(), codes, meta, st.table.cpu(), st.lens.tolist(), st.cu.tolist(), scale, True)
    assert ((block.att[:n].cpu().double() - want[:n]).abs() <= tol[:n]).all()
    A_o, s_o = oracle.quantize_act(block.att.view(block.tokens, -1).cpu().numpy())
    assert _close(block.out, oracle.gemm_w4w8a8(A_o, s_o, oo))


@pytest.mark.parametrize("kind", [torch.float16, torch.float32])
@pytest.mark.parametrize("Hq,H,D,page", [(8, 2, 64, 16), (6, 3, 128, 64)])
def test_prompts_then_decode_steps(dev, kind, Hq, H, D, page):
    K, B = 512, 3
    qkv, oq = _packed(wl.Linear(f"ab_qkv_{Hq}_{D}", 1, (Hq + 2 * H) * D, K, ((0, (Hq + 2 * H) * D, 40),), 4), dev)
    o, oo = _packed(wl.Linear(f"ab_o_{Hq}_{D}", 1, K, Hq * D, ((0, K, 26),), 4), dev)
    g = torch.Generator(device="cuda").manual_seed(7)
    w = (1 + 0.1 * torch.randn(K, generator=g, device=dev)).half()
    cache = mx.kv4_cache(40, H, D, page, dev)
    rope = mx.rope_table(256, D, 10000.0, dev)
    width, scale = -(-200 // page) + 1, D ** -0.5

    # ---- prompts of different lengths, padded to 100 tokens (the tiled GEMM)
    st = _State(B, 40, width, 100, dev)
    st.new.copy_(torch.tensor([37, 0, 52], dtype=torch.int32))
    block = AttentionBlock(w, qkv, o, Hq, cache, rope, 100, B, 52, width)
    r = torch.randn((100, K), generator=g, device=dev).to(kind)
    before = r.clone()
    st.assign(page)
    block.run(r, st.table, st.lens, st.cu, st.slots, st.pos)
    mx.sync_status()
    assert int(st.status) == 0 and torch.equal(r, before)
    _check_stages(block, st, before, None, r, w, oq, oo, 89, scale)

    # ---- decode steps: the same cache, now one token of each request (the few-token kernel), with the residual
    # update of the block before, eagerly once and then as a graph
    st.resize(B, dev)
    st.new.fill_(1)
    step = AttentionBlock(w, qkv, o, Hq, cache, rope, B, B, 1, width)
    r, x = torch.zeros((B, K), dtype=kind, device=dev), torch.zeros((B, K), dtype=torch.float16, device=dev)

    def one():
        st.assign(page)
        step.run(r, st.table, st.lens, st.cu, st.slots, st.pos, x)

    def feed():
        r.copy_(torch.randn((B, K), generator=g, device=dev))
        x.copy_(torch.randn((B, K), generator=g, device=dev))
        return r.clone()

    before = feed()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one()
    torch.cuda.current_stream().wait_stream(side)
    mx.sync_status()
    _check_stages(step, st, before, x, r, w, oq, oo, B, scale)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one()
    for _ in range(20):
        before = feed()
        graph.replay()
    mx.sync_status()
    assert int(st.status) == 0 and st.lens.tolist() == [58, 21, 73]
    _check_stages(step, st, before, x, r, w, oq, oo, B, scale)
    out = step.out.clone()
    # the last step again, eagerly, from the same lengths: the same bits
    st.lens -= 1
    r.copy_(before)
    one()
    mx.sync_status()
    assert torch.equal(out, step.out)


def test_shapes_that_do_not_fit_are_refused(dev):
    p = mx.empty_packed(512, 256, 0, dev)
    o = mx.empty_packed(256, 256, 0, dev)
    w = torch.ones(256, dtype=torch.float16, device=dev)
    cache = mx.kv4_cache(2, 2, 64, 16, dev)
    AttentionBlock(w, p, o, 4, cache, None, 1, 1, 1, 2)
    with pytest.raises(ValueError):
        AttentionBlock(w, p, o, 8, cache, None, 1, 1, 1, 2)
    with pytest.raises(ValueError):
        AttentionBlock(w, p, p, 4, cache, None, 1, 1, 1, 2)
    with pytest.raises(ValueError):
        AttentionBlock(w, p, o, 4, cache, None, 0, 1, 1, 2)
