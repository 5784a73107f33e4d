"""The residual norms between the linears (mixllm_residual_norm) and the way
back from int8 codes to fp16 (mixllm_dequantize_act)."""
from __future__ import annotations

import torch

from . import _lib
from ._call import allocating, call, need, on_cuda, ptr, rows

_F16, _F32 = torch.float16, torch.float32


def _norm(r, w, y, A_q, s_a, x, r_out, w_post, gate, scale, eps, stream):
    dev = on_cuda(r, "r")
    if r.dim() != 2 or r.dtype not in (_F16, _F32):
        raise ValueError("r must be an fp16 or fp32 [M, K]")
    M, K = shape = r.shape
    r_stride = rows(r, "r", r.dtype, shape, dev)
    need(w, "w", _F16, (K,), dev)
    x_stride = gate_stride = out_stride = K
    if x is not None:
        x_stride = rows(x, "x", _F16, shape, dev)
    if w_post is not None:
        need(w_post, "w_post", _F16, (K,), dev)
    if gate is not None:
        one = gate.dim() == 1 or gate.shape[0] == 1
        gate = gate.view(1, -1) if gate.dim() == 1 else gate
        gate_stride = rows(gate, "gate", _F16, (1 if one else M, K), dev)
        gate_stride = 0 if one else gate_stride
    if r_out is not None:
        out_stride = rows(r_out, "r_out", r.dtype, shape, dev)
    if y is not None:
        need(y, "y", _F16, shape, dev)
    if A_q is not None:
        need(A_q, "A_q", torch.int8, shape, dev)
        need(s_a, "s_a", _F32, (M, K // _lib.GROUP), dev)
    call("mixllm_residual_norm", dev, stream, ptr(r), r_stride, r.dtype is _F32, ptr(x), x_stride, ptr(w_post),
         ptr(gate), gate_stride, scale, ptr(r_out), out_stride, ptr(w), eps, M, K, ptr(y), ptr(A_q), ptr(s_a))


def residual_norm_into(r, w, y, x=None, r_out=None, w_post=None, gate=None, scale: float = 1.0, eps: float = 1e-5,
                       stream=None):
    """r' = r + scale * gate * norm(x, w_post) into r_out (which may be r), and
    y = fp16(norm(r', w)).  r and r_out fp16 or fp32 [M, K]; x fp16 [M, K], the
    output of a block, or None (then r' = r); w_post fp16 [K] for a norm after
    the block, or None; gate fp16 [M, K], [1, K] or [K], or None."""
    _norm(r, w, y, None, None, x, r_out, w_post, gate, scale, eps, stream)


def residual_norm_quantize_into(r, w, A_q, s_a, x=None, r_out=None, w_post=None, gate=None, scale: float = 1.0,
                                eps: float = 1e-5, stream=None, y=None):
    """residual_norm_into with y's codes and scales, those of quantize_act(y),
    for the linear that follows (gemm_w4w8a8); y itself only where given."""
    _norm(r, w, y, A_q, s_a, x, r_out, w_post, gate, scale, eps, stream)


def dequantize_act_into(A_q, s_a, X, stream=None):
    """X fp16 [M, K] = A_q * s_a (mixllm_dequantize_act)."""
    dev = on_cuda(A_q, "A_q")
    M, K = shape = A_q.shape
    need(A_q, "A_q", torch.int8, shape, dev)
    need(s_a, "s_a", _F32, (M, K // _lib.GROUP), dev)
    need(X, "X", _F16, shape, dev)
    call("mixllm_dequantize_act", dev, stream, ptr(A_q), ptr(s_a), M, K, _lib.GROUP, ptr(X))


def dequantize_act(A_q, s_a, stream=None) -> torch.Tensor:
    """A_q int8 [M, K], s_a fp32 [M, K/128] -> fp16 [M, K]."""
    with allocating(stream):
        X = torch.empty(A_q.shape, dtype=_F16, device=A_q.device)
    dequantize_act_into(A_q, s_a, X, stream)
    return X
