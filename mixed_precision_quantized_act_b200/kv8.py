"""The paged KV cache in 8 bits and the attention over it (mixllm_kv8_*): the
write (norm, rotation and quantization fused), the read-back and the attention.
Pages and slots are those of the 4-bit cache (kv4_assign_into)."""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from ._call import allocating, call, need, on_cuda, ptr, rows
from .norm import turn

_F16, _F32, _I32, _I64 = torch.float16, torch.float32, torch.int32, torch.int64
KV8_BLOCK = 16  # tokens of one scale


@dataclass
class KV8Cache:
    """A cache of pages: codes uint8 [pages, 2, kv_heads, page_size, head_dim]
    (keys, values; 128 stands for zero) and scales fp32 [pages, 2, kv_heads,
    page_size / 16], one for each block of 16 tokens of a head."""
    codes: torch.Tensor
    scales: torch.Tensor

    def __post_init__(self):
        if self.codes.dim() != 5 or self.codes.shape[1] != 2:
            raise ValueError("codes must be a uint8 [pages, 2, kv_heads, page_size, head_dim]")
        self.index = on_cuda(self.codes, "codes")
        self.pages, _, self.kv_heads, self.page_size, self.head_dim = self.codes.shape
        need(self.codes, "codes", torch.uint8, self.codes.shape, self.index)
        need(self.scales, "scales", _F32, (*self.codes.shape[:3], self.page_size // KV8_BLOCK), self.index)
        self.device = self.codes.device

    def _args(self):
        return (self.codes.data_ptr(), self.scales.data_ptr(), self.pages, self.kv_heads, self.head_dim, self.page_size)

    def nbytes(self) -> int:
        return self.codes.numel() + 4 * self.scales.numel()


def kv8_cache(pages: int, kv_heads: int, head_dim: int, page_size: int = 64, device="cuda") -> KV8Cache:
    """An empty cache of `pages` pages."""
    shape = (pages, 2, kv_heads, page_size)
    return KV8Cache(torch.full(shape + (head_dim,), 128, dtype=torch.uint8, device=device),
                    torch.zeros(shape[:3] + (page_size // KV8_BLOCK,), dtype=_F32, device=device))


def kv8_append_into(k, v, slots, cache: KV8Cache, q=None, q_out=None, positions=None, rope=None, w_q=None, w_k=None,
                    eps: float = 1e-6, stream=None):
    """Quantizes k and v fp16 [T, kv_heads, head_dim] into their slots int64
    [T] (negative: skipped; the tokens of a block of 16 follow one another, with
    only skipped ones between them, within 16 places of the list); with w_k, w_q
    fp16 [head_dim] every key and query head is normalized first, with rope fp32
    [max_pos, rotary] and positions int32 [T] rotated: q fp16 [T, q_heads,
    head_dim] into q_out (which may be q).  A block's scale grows with its tokens,
    and its older rows are re-coded then (mixllm_kv8_append).  Rows may be strided:
    slices of one qkv output serve."""
    dev = cache.index
    T = slots.shape[0]
    D = cache.head_dim
    shape = (T, cache.kv_heads, D)
    if q is not None and q_out is None:
        raise ValueError("q needs q_out")
    need(slots, "slots", _I64, (T,), dev)
    k_stride, v_stride = rows(k, "k", _F16, shape, dev), rows(v, "v", _F16, shape, dev)
    q_heads = q_stride = out_stride = 0
    if q is not None:
        q_heads = q.shape[1]
        q_stride = rows(q, "q", _F16, (T, q_heads, D), dev)
        out_stride = rows(q_out, "q_out", _F16, (T, q_heads, D), dev)
    max_pos, rotary = turn(D, T, w_q, w_k, positions, rope, dev)
    call("mixllm_kv8_append", dev, stream, *cache._args(), ptr(slots), T, ptr(k), k_stride, ptr(v), v_stride, ptr(q),
         q_stride, q_heads, ptr(q_out), out_stride, ptr(w_q), ptr(w_k), eps, ptr(positions), ptr(rope), max_pos, rotary)


def kv8_read_into(slots, cache: KV8Cache, k_out, v_out, stream=None):
    """The cached keys and values of slots int64 [T] into fp16
    [T, kv_heads, head_dim] tensors (mixllm_kv8_read)."""
    dev = cache.index
    T = slots.shape[0]
    shape = (T, cache.kv_heads, cache.head_dim)
    need(slots, "slots", _I64, (T,), dev)
    need(k_out, "k_out", _F16, shape, dev)
    need(v_out, "v_out", _F16, shape, dev)
    call("mixllm_kv8_read", dev, stream, *cache._args(), ptr(slots), T, ptr(k_out), ptr(v_out))


def kv8_attention_workspace_bytes(requests: int, max_q: int, q_heads: int, kv_heads: int, head_dim: int,
                                  page_size: int, table_width: int) -> int:
    out = ctypes.c_size_t(0)
    _lib._check(_lib.load().mixllm_kv8_attention_workspace_bytes(requests, max_q, q_heads, kv_heads, head_dim,
                                                                 page_size, table_width, ctypes.byref(out)),
                "mixllm_kv8_attention_workspace_bytes")
    return out.value


def kv8_attention_workspace(requests: int, max_q: int, q_heads: int, cache: KV8Cache,
                            table_width: int) -> torch.Tensor:
    """A zero-filled workspace for kv8_attention_into with these sizes (calls
    leave its counters at zero; calls that overlap in time must not share one).
    Filled on the current stream: a first call on another has to wait for it."""
    n = kv8_attention_workspace_bytes(requests, max_q, q_heads, cache.kv_heads, cache.head_dim, cache.page_size,
                                      table_width)
    return torch.zeros(max(256, n), dtype=torch.uint8, device=cache.device)


def kv8_attention_into(q, cache: KV8Cache, block_table, seq_lens, cu_q, max_q: int, out, workspace, scale=None,
                       causal: bool = True, lse=None, stream=None):
    """Attention of ragged queries over the cache (mixllm_kv8_attention): rows
    cu_q[b]:cu_q[b+1] of q fp16 [T, q_heads, head_dim] (at most max_q of them)
    against the seq_lens[b] tokens in the pages of block_table's row b.  scale:
    1 / sqrt(head_dim) when None.  lse: fp32 [T, q_heads] or None."""
    dev = cache.index
    T, q_heads = q.shape[0], q.shape[1]
    B = seq_lens.shape[0]
    shape = (T, q_heads, cache.head_dim)
    q_stride = rows(q, "q", _F16, shape, dev)
    out_stride = rows(out, "out", _F16, shape, dev)
    width = block_table.shape[1]
    table_stride = rows(block_table, "block_table", _I32, (B, width), dev)
    need(seq_lens, "seq_lens", _I32, (B,), dev)
    need(cu_q, "cu_q", _I32, (B + 1,), dev)
    need(workspace, "workspace", torch.uint8, (workspace.shape[0],), dev)
    if lse is not None:
        need(lse, "lse", _F32, (T, q_heads), dev)
    call("mixllm_kv8_attention", dev, stream, ptr(q), q_stride, T, q_heads, *cache._args(), ptr(block_table),
         table_stride, width, ptr(seq_lens), ptr(cu_q), B, max_q,
         cache.head_dim ** -0.5 if scale is None else scale, causal, ptr(out), out_stride, ptr(lse), ptr(workspace),
         workspace.shape[0])


def kv8_attention(q, cache: KV8Cache, block_table, seq_lens, cu_q, max_q: int, scale=None, causal: bool = True,
                  workspace=None, stream=None) -> torch.Tensor:
    """kv8_attention_into with a fresh output and, unless given, workspace.
    Rows of q outside every request come back as zeros.  With a stream, both
    are allocated on it."""
    with allocating(stream):
        out = torch.zeros_like(q, memory_format=torch.contiguous_format)
        if workspace is None:
            workspace = kv8_attention_workspace(seq_lens.shape[0], max_q, q.shape[1], cache, block_table.shape[1])
    kv8_attention_into(q, cache, block_table, seq_lens, cu_q, max_q, out, workspace, scale, causal, None, stream)
    return out
