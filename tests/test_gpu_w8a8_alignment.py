"""Outputs that no 16-byte store could take, in every kernel of the 8-bit product
that writes whole tiles.  GPU only."""
import pytest

torch = pytest.importorskip("torch")

import mixed_precision_quantized_act_b200 as mx  # noqa: E402
from tests.test_gpu_w8a8 import _close, _rng, _want, _weights, dev  # noqa: E402,F401

pytestmark = pytest.mark.gpu


# K is one chunk of 128, which no plan can cut into shares: a block has its whole tile and writes it by way of shared
# memory, 16 bytes at a time where N and the address allow.  Tiles of 16, 32 and 64 tokens; two blocks on a tile of 128
# and of 256 tokens.
@pytest.mark.parametrize("M,N", [(1, 1024), (16, 14336), (20, 1024), (40, 1024), (64, 40960), (100, 10240), (300, 8192),
                                 (1000, 8200)])
@pytest.mark.parametrize("K", [48, 128])
def test_whole_tiles_of_any_alignment(dev, M, N, K):  # noqa: F811
    p = _weights(dev, N, K, 2)
    g = _rng(dev, M)
    A = torch.randint(-128, 128, (M, K), generator=g, device=dev, dtype=torch.int8)
    s_a = torch.rand(M, generator=g, device=dev) / 100
    want, tol = _want(A, s_a, p)
    room = torch.full((M * N + 32,), 77.0, dtype=torch.float16, device=dev)
    for off in (0, 1, 2, 3, 4, 8, 12):  # elements of two bytes behind a 256-byte boundary
        Y = room[off:off + M * N].view(M, N)
        mx.w8a8_gemm_into(A, s_a, p, Y)
        mx.sync_status()
        _close(Y, want, tol)
        assert (room[:off] == 77).all() and (room[off + M * N:] == 77).all()
        room.fill_(77)
