"""The paged KV cache in 4 bits and the attention over it (mixllm_kv4_*): pages
and slots of a step's tokens, the write (rotation and quantization fused), the
read-back and the attention."""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from ._call import allocating, call, need, on_cuda, ptr, rows

_F16, _F32, _I32, _I64 = torch.float16, torch.float32, torch.int32, torch.int64


@dataclass
class KV4Cache:
    """A cache of pages: codes uint8 [pages, 2, kv_heads, page_size,
    head_dim / 2] (keys, values) and meta int32 [pages, 2, kv_heads,
    page_size] (fp16 scale in the low half, zero point above it)."""
    codes: torch.Tensor
    meta: torch.Tensor

    def __post_init__(self):
        if self.codes.dim() != 5 or self.codes.shape[1] != 2:
            raise ValueError("codes must be a uint8 [pages, 2, kv_heads, page_size, head_dim / 2]")
        self.index = on_cuda(self.codes, "codes")
        need(self.codes, "codes", torch.uint8, self.codes.shape, self.index)
        need(self.meta, "meta", _I32, self.codes.shape[:4], self.index)
        self.device = self.codes.device
        self.pages, _, self.kv_heads, self.page_size, half = self.codes.shape
        self.head_dim = 2 * half

    def _args(self):
        return (self.codes.data_ptr(), self.meta.data_ptr(), self.pages, self.kv_heads, self.head_dim, self.page_size)

    def nbytes(self) -> int:
        return self.codes.numel() + 4 * self.meta.numel()


def kv4_cache(pages: int, kv_heads: int, head_dim: int, page_size: int = 64, device="cuda") -> KV4Cache:
    """An empty cache of `pages` pages."""
    shape = (pages, 2, kv_heads, page_size)
    return KV4Cache(torch.zeros(shape + (head_dim // 2,), dtype=torch.uint8, device=device),
                    torch.zeros(shape, dtype=_I32, device=device))


def rope_table(max_pos: int, rotary: int, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """fp32 [max_pos, rotary]: cosines, then sines, of pos * theta^(-2i/rotary)
    (the angles in fp64).  An offline step."""
    inv = theta ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)
    angle = torch.outer(torch.arange(max_pos, dtype=torch.float64), inv)
    return torch.cat((angle.cos(), angle.sin()), 1).to(_F32).to(device)


def kv4_assign_into(ctx_lens, new_lens, block_table, free_pages, free_count, page_size: int, seq_lens, cu_new, slots,
                    positions, free_left, status, stream=None):
    """Pages and slots of a step's new tokens (mixllm_kv4_assign): request b's
    new_lens[b] tokens behind its ctx_lens[b] cached ones.  Pages it lacks are
    popped from the stack free_pages[:free_count] into its row of block_table.
    seq_lens may be ctx_lens and free_left may be free_count (in place)."""
    dev = on_cuda(ctx_lens, "ctx_lens")
    B = ctx_lens.shape[0]
    T = slots.shape[0]
    one = (1,)
    need(ctx_lens, "ctx_lens", _I32, (B,), dev)
    need(new_lens, "new_lens", _I32, (B,), dev)
    stride = rows(block_table, "block_table", _I32, (B, block_table.shape[1]), dev)
    need(free_pages, "free_pages", _I32, (free_pages.shape[0],), dev)
    need(free_count, "free_count", _I32, one, dev)
    need(seq_lens, "seq_lens", _I32, (B,), dev)
    need(cu_new, "cu_new", _I32, (B + 1,), dev)
    need(slots, "slots", _I64, (T,), dev)
    need(positions, "positions", _I32, (T,), dev)
    need(free_left, "free_left", _I32, one, dev)
    need(status, "status", _I32, one, dev)
    call("mixllm_kv4_assign", dev, stream, ptr(ctx_lens), ptr(new_lens), B, ptr(block_table), stride,
         block_table.shape[1], ptr(free_pages), free_pages.shape[0], ptr(free_count), page_size, ptr(seq_lens),
         ptr(cu_new), ptr(slots), ptr(positions), T, ptr(free_left), ptr(status))


def kv4_append_into(k, v, slots, cache: KV4Cache, q=None, q_out=None, positions=None, rope=None, stream=None):
    """Quantizes k and v fp16 [T, kv_heads, head_dim] into their slots int64
    [T] (negative: skipped); with rope fp32 [max_pos, rotary] and positions
    int32 [T], rotates the keys and q fp16 [T, q_heads, head_dim] (into q_out,
    which may be q) first.  Rows may be strided: slices of one qkv output serve."""
    dev = cache.index
    T = slots.shape[0]
    shape = (T, cache.kv_heads, cache.head_dim)
    if (q is not None and q_out is None) or (rope is not None and positions is None):
        raise ValueError("q needs q_out, and rope positions")
    need(slots, "slots", _I64, (T,), dev)
    k_stride, v_stride = rows(k, "k", _F16, shape, dev), rows(v, "v", _F16, shape, dev)
    q_heads = q_stride = out_stride = max_pos = rotary = 0
    if q is not None:
        q_heads = q.shape[1]
        q_stride = rows(q, "q", _F16, (T, q_heads, cache.head_dim), dev)
        out_stride = rows(q_out, "q_out", _F16, (T, q_heads, cache.head_dim), dev)
    if rope is not None:
        max_pos, rotary = rope.shape
        need(rope, "rope", _F32, rope.shape, dev)
        need(positions, "positions", _I32, (T,), dev)
    call("mixllm_kv4_append", dev, stream, *cache._args(), ptr(slots), T, ptr(k), k_stride, ptr(v), v_stride, ptr(q),
         q_stride, q_heads, ptr(q_out), out_stride, ptr(positions), ptr(rope), max_pos, rotary)


def kv4_read_into(slots, cache: KV4Cache, k_out, v_out, stream=None):
    """The cached keys and values of slots int64 [T] into fp16
    [T, kv_heads, head_dim] tensors (mixllm_kv4_read)."""
    dev = cache.index
    T = slots.shape[0]
    shape = (T, cache.kv_heads, cache.head_dim)
    need(slots, "slots", _I64, (T,), dev)
    need(k_out, "k_out", _F16, shape, dev)
    need(v_out, "v_out", _F16, shape, dev)
    call("mixllm_kv4_read", dev, stream, *cache._args(), ptr(slots), T, ptr(k_out), ptr(v_out))


def kv4_attention_workspace_bytes(requests: int, max_q: int, q_heads: int, kv_heads: int, head_dim: int,
                                  page_size: int, table_width: int) -> int:
    out = ctypes.c_size_t(0)
    _lib._check(_lib.load().mixllm_kv4_attention_workspace_bytes(requests, max_q, q_heads, kv_heads, head_dim,
                                                                 page_size, table_width, ctypes.byref(out)),
                "mixllm_kv4_attention_workspace_bytes")
    return out.value


def kv4_attention_workspace(requests: int, max_q: int, q_heads: int, cache: KV4Cache,
                            table_width: int) -> torch.Tensor:
    """A zero-filled workspace for kv4_attention_into with these sizes (calls
    leave its counters at zero; calls that overlap in time must not share one).
    Filled on the current stream: a first call on another has to wait for it."""
    n = kv4_attention_workspace_bytes(requests, max_q, q_heads, cache.kv_heads, cache.head_dim, cache.page_size,
                                      table_width)
    return torch.zeros(max(256, n), dtype=torch.uint8, device=cache.device)


def kv4_attention_into(q, cache: KV4Cache, block_table, seq_lens, cu_q, max_q: int, out, workspace, scale=None,
                       causal: bool = True, lse=None, stream=None):
    """Attention of ragged queries over the cache (mixllm_kv4_attention): rows
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
    call("mixllm_kv4_attention", dev, stream, ptr(q), q_stride, T, q_heads, *cache._args(), ptr(block_table),
         table_stride, width, ptr(seq_lens), ptr(cu_q), B, max_q,
         cache.head_dim ** -0.5 if scale is None else scale, causal, ptr(out), out_stride, ptr(lse), ptr(workspace),
         workspace.shape[0])


def kv4_attention(q, cache: KV4Cache, block_table, seq_lens, cu_q, max_q: int, scale=None, causal: bool = True,
                  workspace=None, stream=None) -> torch.Tensor:
    """kv4_attention_into with a fresh output and, unless given, workspace.
    Rows of q outside every request come back as zeros.  With a stream, both
    are allocated on it."""
    with allocating(stream):
        out = torch.zeros_like(q, memory_format=torch.contiguous_format)
        if workspace is None:
            workspace = kv4_attention_workspace(seq_lens.shape[0], max_q, q.shape[1], cache, block_table.shape[1])
    kv4_attention_into(q, cache, block_table, seq_lens, cu_q, max_q, out, workspace, scale, causal, None, stream)
    return out
