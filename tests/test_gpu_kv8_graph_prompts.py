"""A prompt's step over the 8-bit cache as a replayed graph: above 512 tokens the
append is two kernels, the second of which starts beside the first.  GPU only."""
import pytest

torch = pytest.importorskip("torch")

import mixed_precision_quantized_act_b200 as mx  # noqa: E402
from tests.test_gpu_kv8 import dev  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [512, 513, 1400])
@pytest.mark.parametrize("in_place", [False, True])
def test_prompts_as_a_graph(dev, T, in_place):  # noqa: F811
    Hq, H, D, page = 16, 2, 128, 64
    pages = -(-T // page) + 1
    g = torch.Generator(device=dev).manual_seed(T)
    randn = lambda *s: torch.randn(s, generator=g, device=dev).half()  # noqa: E731
    w, rope = (1 + 0.1 * randn(D)).half(), mx.rope_table(T, D, device=dev)
    table = torch.randperm(pages, generator=g, device=dev).to(torch.int32)[None]
    at = torch.arange(T, device=dev)
    slots, pos = table[0, at // page].long() * page + at % page, at.to(torch.int32)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    lens, cu = i32([T]), i32([0, T])
    x, q_out, out = torch.zeros((T, Hq + 2 * H, D), device=dev).half(), randn(T, Hq, D), torch.zeros((T, Hq, D), device=dev).half()

    def step(x, cache, q_out, out, ws):
        q, k, v = x.split((Hq, H, H), 1)
        q_out = q if in_place else q_out
        mx.kv8_append_into(k, v, slots, cache, q=q, q_out=q_out, positions=pos, rope=rope, w_q=w, w_k=w)
        mx.kv8_attention_into(q_out, cache, table, lens, cu, T, out, ws)

    cache, plain = (mx.kv8_cache(pages, H, D, page, dev) for _ in range(2))
    ws, ws_plain = (mx.kv8_attention_workspace(1, T, Hq, cache, pages) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, cache, q_out, out, ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(x, cache, q_out, out, ws)
        step(x if not in_place else x.clone(), cache, q_out, out, ws)  # the next step's append follows at once
    for _ in range(6):
        new, want = randn(T, Hq + 2 * H, D), torch.empty_like(out)
        x.copy_(new)
        graph.replay()
        first = new.clone()
        step(first, plain, torch.empty_like(q_out), want, ws_plain)
        if in_place:  # its second step turns what the first left
            step(first, plain, None, want, ws_plain)
        torch.cuda.synchronize()
        assert torch.equal(cache.codes, plain.codes) and torch.equal(cache.scales, plain.scales)
        assert torch.equal(out, want)
    mx.sync_status()
