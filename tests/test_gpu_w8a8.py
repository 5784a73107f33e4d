"""The 8-bit linears on the GPU: weights and activations against the quantizer's
definition, the product against exact integers.  GPU only."""
import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mixed_precision_quantized_act_b200 as mx  # noqa: E402
from tests import kv8_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.load()
    return torch.device("cuda:0")


def _rng(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


def _weights(dev, N, K, seed=0):
    g = _rng(dev, seed)
    codes = torch.randint(-127, 128, (N, K), generator=g, device=dev, dtype=torch.int8)
    return mx.W8Weights(codes, (0.5 + torch.rand(N, generator=g, device=dev)) / K)


def _want(A, s_a, p, bias=None):
    """The product's definition in 64 bits, and the tolerance of each output: one rounding to fp16 (2^-11, half a step
    of 2^-24 below its normal numbers) and, of the terms before the sum with the bias, four of fp32 (the integer as
    fp32, two products, the FMA)."""
    term = A.double() @ p.codes.double().t() * s_a.double()[:, None] * p.s_w.double()
    y = term if bias is None else term + bias.double()
    return y, 2.0 ** -11 * y.abs() + 4 * 2.0 ** -24 * (term.abs() + y.abs()) + 2.0 ** -25


def _close(Y, want, tol):
    off = (Y.double() - want).abs()
    assert (off <= tol).all(), float((off / tol).max())


# a token, a few, one tile of each width and its neighbours, both kernels of prompts; K and N of no tile's multiple
SHAPES = [(1, 1, 16), (1, 129, 128), (3, 300, 144), (16, 4096, 2048), (17, 1000, 1040), (32, 257, 4096), (33, 64, 528),
          (64, 2000, 256), (65, 515, 272), (70, 9000, 640), (128, 8192, 384), (129, 4100, 512), (250, 4096, 1024),
          (257, 8200, 160), (511, 2049, 400), (700, 16384, 208), (1025, 4096, 320), (5, 40000, 64), (40, 38000, 48)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("with_bias", [False, True])
def test_product_of_given_codes(dev, M, N, K, with_bias):
    g = _rng(dev, M + N + K)
    p = _weights(dev, N, K)
    A = torch.randint(-128, 128, (M, K), generator=g, device=dev, dtype=torch.int8)
    s_a = torch.rand(M, generator=g, device=dev) / 100
    bias = torch.randn(N, generator=g, device=dev).half() if with_bias else None
    Y = torch.full((M, N), float("nan"), dtype=torch.float16, device=dev)
    mx.w8a8_gemm_into(A, s_a, p, Y, bias=bias)
    mx.sync_status()
    _close(Y, *_want(A, s_a, p, bias))
    again = torch.full_like(Y, float("nan"))
    mx.w8a8_gemm_into(A, s_a, p, again, bias=bias)
    assert torch.equal(Y.view(torch.int16), again.view(torch.int16))


# one block an SM: whole K, two, three or four shares of it, the last tile of channels full, ragged and of one channel;
# four tokens of which the last are one, and none
ALONE = [(64, 4096, 1024), (33, 3969, 4096), (50, 6000, 784), (61, 6144, 2064), (40, 8193, 2064), (63, 9472, 512),
         (34, 13001, 272), (64, 18944, 400), (49, 5000, 14336), (1, 12300, 1024), (16, 16384, 400), (3, 14337, 4096),
         (32, 4096, 1024), (17, 6000, 784), (25, 13001, 272), (20, 8193, 2064), (31, 18432, 336)]


@pytest.mark.parametrize("M,N,K", ALONE)
@pytest.mark.parametrize("with_bias", [False, True])
def test_some_tokens_of_few_tiles(dev, M, N, K, with_bias):
    test_product_of_given_codes(dev, M, N, K, with_bias)
    test_linear_is_quantizer_and_product(dev, M, N, K)


# two blocks on a tile of 128 tokens, and of 256: the last tile of either side full, ragged, for the first block alone
PAIRS = [(65, 13000, 48), (70, 9600, 640), (127, 9601, 528), (300, 6144, 272), (500, 4096, 1024), (511, 4097, 400),
         (1025, 4096, 2064), (129, 20000, 1040), (700, 16300, 528), (1024, 4096, 4096), (1500, 2177, 144)]


@pytest.mark.parametrize("M,N,K", PAIRS)
@pytest.mark.parametrize("with_bias", [False, True])
def test_many_tokens(dev, M, N, K, with_bias):
    test_product_of_given_codes(dev, M, N, K, with_bias)
    test_linear_is_quantizer_and_product(dev, M, N, K)


def test_a_first_call_within_a_capture():
    """Nothing that the launch asks the runtime for, once a process, is refused while a stream is captured."""
    code = """
import torch, mixed_precision_quantized_act_b200 as mx
mx.load()
p = mx.W8Weights(torch.ones((4096, 1024), dtype=torch.int8, device="cuda"), torch.ones(4096, device="cuda"))
X = torch.full((64, 1024), 0.5, device="cuda").half()
Y, ws = torch.zeros((64, 4096), device="cuda").half(), mx.w8a8_linear_workspace(64, p)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    mx.w8a8_linear_into(X, p, Y, ws)
assert not Y.any()
g.replay()
torch.cuda.synchronize()
assert (Y == 512).all()
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300, cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


@pytest.mark.parametrize("K", [131056, 131056 - 64])
def test_sums_at_the_ends_of_int32(dev, K):
    """128 x 128 x 131056 is just below 2^31."""
    p = mx.W8Weights(torch.full((130, K), -128, dtype=torch.int8, device=dev), torch.full((130,), 2.0 ** -16, device=dev))
    p.codes[1] = 127
    A = torch.full((5, K), -128, dtype=torch.int8, device=dev)
    s_a = torch.full((5,), 2.0 ** -4, device=dev)
    Y = torch.empty((5, 130), dtype=torch.float16, device=dev)
    mx.w8a8_gemm_into(A, s_a, p, Y)
    mx.sync_status()
    _close(Y, *_want(A, s_a, p))


@pytest.mark.parametrize("M,K", [(1, 16), (1, 4096), (7, 144), (600, 2064), (3, 8208), (513, 33000 // 16 * 16), (2, 131056)])
def test_activation_codes(dev, M, K):
    g = _rng(dev, K)
    x = (torch.randn((M, K), generator=g, device=dev) * 10 ** torch.randint(-5, 4, (M, 1), generator=g, device=dev)).half()
    x[0, :16] = torch.arange(16, device=dev).half() - 8  # ties, with the largest at 127 or 254
    if M > 1:
        x[1] = 0
    if M > 2:
        x[2] = torch.randint(-254, 255, (K,), generator=g, device=dev).half() / 2
        x[2, 0] = 127
    A, s = mx.w8a8_quantize(x)
    mx.sync_status()
    q, want = ref.quantize_rows(x.cpu().numpy())
    assert np.array_equal(s.cpu().numpy().view(np.uint32), want.view(np.uint32))
    assert np.array_equal(A.cpu().numpy(), q)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("K", [64, 40000])
def test_rows_that_are_not_finite(dev, bad, K):
    x = torch.ones((3, K), device=dev).half()
    x[1, K - 1] = bad
    A, s = mx.w8a8_quantize(x)
    assert s.isnan().tolist() == [False, True, False] and not A[1].any()
    p = _weights(dev, 40, K)
    Y = mx.w8a8_linear(x, p)
    mx.sync_status()
    assert Y[1].isnan().all() and Y[[0, 2]].isfinite().all()
    p = mx.w8a8_pack(x.float())
    assert p.s_w.isnan().tolist() == [False, True, False] and not p.codes[1].any()


@pytest.mark.parametrize("N,K", [(1, 16), (300, 272), (5, 20000)])
def test_weight_codes(dev, N, K):
    W = torch.randn((N, K), generator=_rng(dev, N), device=dev) * 0.02
    W[0, 3] = 0.5
    p = mx.w8a8_pack(W)
    mx.sync_status()
    q, s = ref.quantize_rows(W.cpu().numpy())
    assert np.array_equal(p.s_w.cpu().numpy().view(np.uint32), s.view(np.uint32)) and np.array_equal(p.codes.cpu().numpy(), q)


@pytest.mark.parametrize("M,N,K", [(1, 515, 144), (40, 1024, 512), (130, 4096, 256), (600, 8192, 512)])
def test_linear_is_quantizer_and_product(dev, M, N, K):
    """Rows of X apart; a workspace of more tokens, dirty, serves."""
    p = _weights(dev, N, K, 1)
    wide = torch.randn((M, K + 24), generator=_rng(dev, M), device=dev).half()
    X = wide[:, 8:8 + K]
    ws = mx.w8a8_linear_workspace(M + 50, p)
    ws.fill_(255)
    Y = torch.full((M, N), float("nan"), dtype=torch.float16, device=dev)
    mx.w8a8_linear_into(X, p, Y, ws)
    A, s_a = mx.w8a8_quantize(X)
    two = torch.empty_like(Y)
    mx.w8a8_gemm_into(A, s_a, p, two)
    mx.sync_status()
    assert torch.equal(Y, two)
    q, s = ref.quantize_rows(X.cpu().numpy())
    _close(Y, *_want(torch.from_numpy(q).to(dev), torch.from_numpy(s).to(dev), p))


@pytest.mark.parametrize("M", [1, 40, 300])
def test_outputs_of_any_alignment(dev, M):
    """A Y that no vector store could take, and outputs beside it left as they were."""
    p = _weights(dev, 1024, 256, 2)
    X = torch.randn((M, 256), generator=_rng(dev, 3), device=dev).half()
    want = mx.w8a8_linear(X, p)
    room = torch.full((M * 1024 + 16,), 77.0, dtype=torch.float16, device=dev)
    for off in (1, 2, 4, 8):
        Y = room[off:off + M * 1024].view(M, 1024)
        mx.w8a8_linear_into(X, p, Y, mx.w8a8_linear_workspace(M, p))
        mx.sync_status()
        assert torch.equal(Y, want)
        assert (room[:off] == 77).all() and (room[off + M * 1024:] == 77).all()
        room.fill_(77)


def test_values_beyond_fp16_become_infinite(dev):
    p = mx.W8Weights(torch.full((8, 64), 127, dtype=torch.int8, device=dev), torch.ones(8, device=dev))
    Y = torch.empty((2, 8), dtype=torch.float16, device=dev)
    mx.w8a8_gemm_into(torch.tensor([[127] * 64, [-127] * 64], dtype=torch.int8, device=dev), torch.ones(2, device=dev), p, Y)
    assert Y.tolist() == [[float("inf")] * 8, [-float("inf")] * 8]


def test_weights_written_by_the_kernel_before(dev):
    """The product may start early; it still sees what the kernels before it on the stream wrote."""
    W = [torch.randn((2048, 512), generator=_rng(dev, i), device=dev) for i in range(2)]
    X = torch.randn((20, 512), generator=_rng(dev, 9), device=dev).half()
    want = [mx.w8a8_linear(X, mx.w8a8_pack(w)) for w in W]
    p = mx.w8a8_pack(W[0])
    ws, Y = mx.w8a8_linear_workspace(20, p), torch.empty((20, 2048), dtype=torch.float16, device=dev)
    A, s_a = mx.w8a8_quantize(X)
    packed = [mx.w8a8_pack(w) for w in W]
    torch.cuda.synchronize()
    for i in range(40):
        p.codes.copy_(packed[i % 2].codes)
        p.s_w.copy_(packed[i % 2].s_w)
        if i % 4 < 2:
            mx.w8a8_linear_into(X, p, Y, ws)
        else:
            mx.w8a8_gemm_into(A, s_a, p, Y)
        assert torch.equal(Y, want[i % 2])


@pytest.mark.parametrize("M", [1, 100, 400])
def test_in_a_graph_and_on_two_streams(dev, M):
    p = _weights(dev, 4096, 512, 4)
    X = [torch.randn((M, 512), generator=_rng(dev, i), device=dev).half() for i in range(2)]
    want = [mx.w8a8_linear(x, p) for x in X]
    x, Y, ws = X[0].clone(), torch.empty_like(want[0]), mx.w8a8_linear_workspace(M, p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mx.w8a8_linear_into(x, p, Y, ws, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.w8a8_linear_into(x, p, Y, ws)
        mx.w8a8_linear_into(x, p, Y, ws)
    for i in range(10):
        x.copy_(X[i % 2])
        graph.replay()
        assert torch.equal(Y, want[i % 2])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty_like(Y) for _ in range(2)]
    spaces = [mx.w8a8_linear_workspace(M, p) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, x, y, w in zip(streams, X, outs, spaces):
            mx.w8a8_linear_into(x, p, y, w, stream=s)
    torch.cuda.synchronize()
    mx.sync_status()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_nothing_to_do(dev):
    p = _weights(dev, 32, 64)
    assert mx.w8a8_linear(torch.empty((0, 64), dtype=torch.float16, device=dev), p).shape == (0, 32)
    none = mx.W8Weights(torch.empty((0, 64), dtype=torch.int8, device=dev), torch.empty(0, device=dev))
    assert mx.w8a8_linear(torch.ones((3, 64), dtype=torch.float16, device=dev), none).shape == (3, 0)
    assert mx.w8a8_pack(torch.empty((0, 64), device=dev)).N == 0
    mx.sync_status()


def test_bindings_check_their_tensors(dev):
    p = _weights(dev, 32, 64)
    X, Y, ws = torch.ones((2, 64), device=dev).half(), torch.empty((2, 32), device=dev).half(), mx.w8a8_linear_workspace(2, p)
    for bad in (lambda: mx.w8a8_linear_into(X.float(), p, Y, ws), lambda: mx.w8a8_linear_into(X[:, :48], p, Y, ws),
                lambda: mx.w8a8_linear_into(X, p, Y[:1], ws), lambda: mx.w8a8_linear_into(X, p, Y.t().contiguous().t(), ws),
                lambda: mx.w8a8_linear_into(X, p, Y, ws, bias=torch.ones(32, device=dev)),
                lambda: mx.w8a8_linear_into(X.cpu(), p, Y, ws), lambda: mx.w8a8_linear_into(X.t().contiguous().t(), p, Y, ws),
                lambda: mx.W8Weights(p.codes, p.s_w[:5]), lambda: mx.W8Weights(p.codes.float(), p.s_w),
                lambda: mx.W8Weights(p.codes.cpu(), p.s_w.cpu()), lambda: mx.w8a8_pack(torch.ones((2, 32))),
                lambda: mx.w8a8_linear_into(X, p, Y, ws.float())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(mx.MixLLMError):
        mx.w8a8_linear_into(X, p, Y, ws[:100])
    with pytest.raises(mx.MixLLMError):
        mx.w8a8_pack(torch.ones((4, 40), device=dev))  # K
