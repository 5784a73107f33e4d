"""The linear layer in 8-bit integers with a scale per token and per output
channel (mixllm_w8a8_*): weights, activations and the product."""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from ._call import allocating, call, need, on_cuda, ptr, rows

_F16, _F32, _I8 = torch.float16, torch.float32, torch.int8


@dataclass
class W8Weights:
    """One layer's weights: codes int8 [N, K] and a scale fp32 [N] for each
    output channel."""
    codes: torch.Tensor
    s_w: torch.Tensor

    def __post_init__(self):
        if self.codes.dim() != 2:
            raise ValueError("codes must be an int8 [N, K]")
        self.index = on_cuda(self.codes, "codes")
        self.device = self.codes.device
        self.N, self.K = self.codes.shape
        need(self.codes, "codes", _I8, self.codes.shape, self.index)
        need(self.s_w, "s_w", _F32, (self.N,), self.index)

    def buffers(self):
        return self.codes, self.s_w

    def nbytes(self) -> int:
        return self.codes.numel() + 4 * self.s_w.numel()


def w8a8_pack(W, stream=None) -> W8Weights:
    """W fp32 [N, K] as 8-bit codes with a scale per channel (an offline step)."""
    dev = on_cuda(W, "W")
    N, K = W.shape
    need(W, "W", _F32, (N, K), dev)
    with allocating(stream):
        p = W8Weights(torch.empty((N, K), dtype=_I8, device=W.device), torch.empty(N, dtype=_F32, device=W.device))
    call("mixllm_w8a8_pack", dev, stream, ptr(W), N, K, ptr(p.codes), ptr(p.s_w))
    return p


def w8a8_quantize_into(X, A_q, s_a, stream=None):
    """X fp16 [M, K] (rows may be strided) into A_q int8 [M, K] and s_a fp32 [M],
    one scale per token."""
    dev = on_cuda(X, "X")
    M, K = X.shape
    stride = rows(X, "X", _F16, (M, K), dev)
    need(A_q, "A_q", _I8, (M, K), dev)
    need(s_a, "s_a", _F32, (M,), dev)
    call("mixllm_w8a8_quantize", dev, stream, ptr(X), stride, M, K, ptr(A_q), ptr(s_a))


def w8a8_quantize(X, stream=None):
    """X fp16 [M, K] -> (A_q int8 [M, K], s_a fp32 [M])."""
    with allocating(stream):
        A_q = torch.empty(X.shape, dtype=_I8, device=X.device)
        s_a = torch.empty(X.shape[:1], dtype=_F32, device=X.device)
    w8a8_quantize_into(X, A_q, s_a, stream)
    return A_q, s_a


def w8a8_linear_workspace_bytes(M: int, K: int, N: int) -> int:
    out = ctypes.c_size_t(0)
    _lib._check(_lib.load().mixllm_w8a8_linear_workspace_bytes(M, K, N, ctypes.byref(out)),
                "mixllm_w8a8_linear_workspace_bytes")
    return out.value


def w8a8_linear_workspace(M: int, p: W8Weights) -> torch.Tensor:
    """A workspace for w8a8_linear_into with up to M tokens (calls that overlap
    in time must not share one; it needs no initial value)."""
    n = w8a8_linear_workspace_bytes(M, p.K, p.N)
    return torch.empty(max(256, n), dtype=torch.uint8, device=p.device)


def _checked(M, p, Y, bias):
    need(Y, "Y", _F16, (M, p.N), p.index)
    if bias is not None:
        need(bias, "bias", _F16, (p.N,), p.index)


def w8a8_gemm_into(A_q, s_a, p: W8Weights, Y, bias=None, stream=None):
    """Y fp16 [M, N] from A_q int8 [M, K] and s_a fp32 [M] (mixllm_w8a8_gemm);
    bias fp16 [N] or None."""
    M = A_q.shape[0]
    need(A_q, "A_q", _I8, (M, p.K), p.index)
    need(s_a, "s_a", _F32, (M,), p.index)
    _checked(M, p, Y, bias)
    call("mixllm_w8a8_gemm", p.index, stream, ptr(A_q), ptr(s_a), M, p.K, ptr(p.codes), ptr(p.s_w), p.N, ptr(bias),
         ptr(Y))


def w8a8_linear_into(X, p: W8Weights, Y, workspace, bias=None, stream=None):
    """Y fp16 [M, N] from X fp16 [M, K], whose rows may be strided, quantized on
    the way (mixllm_w8a8_linear); bias fp16 [N] or None."""
    M = X.shape[0]
    stride = rows(X, "X", _F16, (M, p.K), p.index)
    _checked(M, p, Y, bias)
    need(workspace, "workspace", torch.uint8, (workspace.shape[0],), p.index)
    call("mixllm_w8a8_linear", p.index, stream, ptr(X), stride, M, p.K, ptr(p.codes), ptr(p.s_w), p.N, ptr(bias),
         ptr(Y), ptr(workspace), workspace.shape[0])


def w8a8_linear(X, p: W8Weights, bias=None, workspace=None, stream=None) -> torch.Tensor:
    """w8a8_linear_into with a fresh output and, unless given, workspace, both
    allocated on the stream."""
    with allocating(stream):
        Y = torch.empty((X.shape[0], p.N), dtype=_F16, device=p.device)
        if workspace is None:
            workspace = w8a8_linear_workspace(X.shape[0], p)
    w8a8_linear_into(X, p, Y, workspace, bias, stream)
    return Y
