"""The linears of one decoder layer as a single CUDA graph, and the layer's
attention half around two of them.

A Llama decoder layer runs four W4.4A8 linears -- fused qkv, o_proj, fused
gate_up and down -- each as activation quantization followed by the fused
GEMM (MLSys 2026 talk notes on MixLLM, notes.yuuk.io, §探索の特性: the
per-layer view of the method's kernels).  The attention core, the norms and
the SwiGLU between them are not part of the method and are not run by
`LinearChain`: each linear reads its own input buffer.  `AttentionBlock` runs
what a served model needs between and around the first two linears.

`LinearChain` holds the packed weights and every intermediate buffer of such
a chain, runs it eagerly, and captures it once into a CUDA graph so that a
replay issues all of its kernels with one launch from the host.  For M <= 64
each linear is one mixllm_linear_small_m call (by default; fused=False keeps
quantize_act and the few-token GEMM as two calls): where the plan allows, the
GEMV quantizes its own slice of X and the layer is a single kernel.  Buffers
are allocated once, at construction; a replay allocates nothing.
"""
from dataclasses import dataclass
from typing import List, Optional

import torch

from . import _lib, kv4, norm


@dataclass
class _Stage:
    p: _lib.PackedLinear
    X: torch.Tensor      # fp16 [M, K] input (filled by the caller)
    A_q: torch.Tensor    # int8 [M, K]
    s_a: torch.Tensor    # fp32 [M, K/128]
    Y: torch.Tensor      # fp16 [M, N] output
    ws: Optional[torch.Tensor]  # few-token workspace, or None
    lws: Optional[torch.Tensor]  # workspace of the fused few-token layer, or None


class LinearChain:
    """A fixed sequence of W4.4A8 linears over one batch of M tokens."""

    def __init__(self, packed: List[_lib.PackedLinear], M: int, device, fused: bool = True):
        self.M = M
        self.fused = fused
        self.device = torch.device(device)
        self.stages: List[_Stage] = []
        for p in packed:
            X = torch.zeros((M, p.K), dtype=torch.float16, device=self.device)
            A_q = torch.empty((M, p.K), dtype=torch.int8, device=self.device)
            s_a = torch.empty((M, p.K // _lib.GROUP), dtype=torch.float32, device=self.device)
            Y = torch.empty((M, p.N), dtype=torch.float16, device=self.device)
            small = 0 < M <= _lib.SMALL_M_MAX
            ws = _lib.small_m_workspace(M, p, self.device) if small else None
            lws = _lib.linear_small_m_workspace(M, p, self.device) if small and fused else None
            self.stages.append(_Stage(p, X, A_q, s_a, Y, ws, lws))
        self.graph: Optional[torch.cuda.CUDAGraph] = None

    @property
    def inputs(self) -> List[torch.Tensor]:
        return [s.X for s in self.stages]

    @property
    def outputs(self) -> List[torch.Tensor]:
        return [s.Y for s in self.stages]

    def launches(self) -> int:
        """Kernels one run issues: one per linear whose GEMV quantizes its own
        activations (the fused workspace is no larger than the GEMM's alone),
        two otherwise."""
        n = 0
        for s in self.stages:
            fused = s.lws is not None and s.lws.numel() == max(
                256, _lib.small_m_workspace_bytes(self.M, s.p.K, s.p.N4, s.p.N8))
            n += 1 if fused else 2
        return n

    def ops(self) -> int:
        return sum(2 * self.M * s.p.N * s.p.K for s in self.stages)

    def run(self, stream=None):
        """Every stage, eagerly, on `stream` (default: the current stream)."""
        for s in self.stages:
            if s.lws is not None:
                _lib.linear_small_m_into(s.X, s.p, s.Y, s.lws, stream)
                continue
            _lib.quantize_act_into(s.X, s.A_q, s.s_a, stream)
            if s.ws is not None:
                _lib.gemm_w4w8a8_small_m_into(s.A_q, s.s_a, s.p, s.Y, s.ws, stream)
            else:
                _lib.gemm_w4w8a8_into(s.A_q, s.s_a, s.p, s.Y, stream)

    def capture(self):
        """Record the chain into a CUDA graph (after one eager warm-up run on a
        side stream, which also builds the library's cached descriptors)."""
        side = torch.cuda.Stream(device=self.device)
        side.wait_stream(torch.cuda.current_stream(self.device))
        with torch.cuda.stream(side):
            self.run()
        torch.cuda.current_stream(self.device).wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.run()
        self.graph = g
        return g

    def replay(self):
        if self.graph is None:
            self.capture()
        self.graph.replay()

    def release(self):
        self.graph = None


class AttentionBlock:
    """The attention half of one decoder layer over a 4-bit paged cache:

        r <- r + x;  y = norm(r);  q, k, v = qkv(y);  q, k <- rotated;
        cache <- k, v in 4 bits;  out = o_proj(attention(q, cache))

    for up to `tokens` tokens of up to `requests` requests at a time.  x is the
    output of the block before (the residual update and its norm are one kernel
    with the quantization for the qkv linear); `out` is this one's, for the block
    after to add.  Buffers are allocated once, and ready for any stream when the
    constructor returns; `run` allocates nothing and can be captured into a graph,
    lengths and slots being device tensors (kv4_assign_into).
    """

    def __init__(self, w_norm: torch.Tensor, qkv: _lib.PackedLinear, o_proj: _lib.PackedLinear, q_heads: int,
                 cache: kv4.KV4Cache, rope: Optional[torch.Tensor], tokens: int, requests: int, max_q: int,
                 table_width: int, eps: float = 1e-5):
        H, D = cache.kv_heads, cache.head_dim
        _lib._require(qkv.N == (q_heads + 2 * H) * D, "qkv must have (q_heads + 2 kv_heads) x head_dim channels")
        _lib._require(o_proj.K == q_heads * D and o_proj.N == qkv.K, "o_proj must lead from the heads to qkv's inputs")
        _lib._require(tokens > 0, "need room for at least one token")
        dev = cache.device
        _lib._require(all(t.device == dev for p in (qkv, o_proj) for t in p.buffers()),
                      f"the packed linears must be on the cache's device, {dev}")
        self.w_norm, self.qkv, self.o_proj, self.cache, self.rope, self.eps = w_norm, qkv, o_proj, cache, rope, eps
        self.q_heads, self.tokens, self.max_q = q_heads, tokens, max_q
        self.A_q = torch.empty((tokens, qkv.K), dtype=torch.int8, device=dev)
        self.s_a = torch.empty((tokens, qkv.K // _lib.GROUP), dtype=torch.float32, device=dev)
        self.heads = torch.empty((tokens, q_heads + 2 * H, D), dtype=torch.float16, device=dev)
        self.q = torch.zeros((tokens, q_heads, D), dtype=torch.float16, device=dev)
        self.att = torch.zeros((tokens, q_heads, D), dtype=torch.float16, device=dev)
        self.out = torch.empty((tokens, o_proj.N), dtype=torch.float16, device=dev)
        self.few = tokens <= _lib.SMALL_M_MAX
        self.ws_qkv = _lib.small_m_workspace(tokens, qkv, dev) if self.few else None
        self.ws_o = _lib.linear_workspace(tokens, o_proj, dev)
        self.ws_att = kv4.kv4_attention_workspace(requests, max_q, q_heads, cache, table_width)
        # the fills above went to the current stream, and `run` may be given any: its kernels' counters start at zero
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(dev).synchronize()

    def run(self, r: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, cu_q: torch.Tensor,
            slots: torch.Tensor, positions: torch.Tensor, x: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """One pass: r fp16 or fp32 [tokens, K] is updated in place when x is
        given; returns the output buffer fp16 [tokens, K].  seq_lens counts the
        new tokens (behind those cached); rows behind cu_q's last entry are padding
        and their outputs of no meaning."""
        with torch.cuda.device(self.cache.device):  # whatever the current device is
            H = self.cache.kv_heads
            norm.residual_norm_quantize_into(r, self.w_norm, self.A_q, self.s_a, x=x, r_out=None if x is None else r,
                                             eps=self.eps, stream=stream)
            Y = self.heads.view(self.tokens, -1)
            if self.few:
                _lib.gemm_w4w8a8_small_m_into(self.A_q, self.s_a, self.qkv, Y, self.ws_qkv, stream)
            else:
                _lib.gemm_w4w8a8_into(self.A_q, self.s_a, self.qkv, Y, stream)
            q, k, v = self.heads.split((self.q_heads, H, H), 1)
            kv4.kv4_append_into(k, v, slots, self.cache, q=q, q_out=self.q, positions=positions, rope=self.rope,
                                stream=stream)
            kv4.kv4_attention_into(self.q, self.cache, block_table, seq_lens, cu_q, self.max_q, self.att, self.ws_att,
                                   stream=stream)
            _lib.linear_into(self.att.view(self.tokens, -1), self.o_proj, self.out, self.ws_o, stream)
        return self.out
