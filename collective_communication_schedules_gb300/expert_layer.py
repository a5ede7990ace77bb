"""A gated expert layer over simulated ranks on one GPU, forward and backward.

HOCCL section 2.1 and Table 1: expert-parallel token dispatch and combine are
all-to-all traffic around the experts' products.  This driver runs the whole
layer with the dispatch and combine fused with their exchange (include/hoc_ep.h)
and the products between them (include/hoc_layer.h):

    recv = dispatch(x, ids)                      rows of each expert, by source
    h    = silu(recv W_gate^T) * (recv W_up^T)   w_up[d]: [experts, 2 * ffn, hidden], gates first
    out  = h W_down^T                            w_down[d]: [experts, hidden, ffn]
    y    = combine(out, gate)                    gate-weighted sum of a token's rows

With rows of 8 bits (include/hoc_block.h) the dispatch moves those, about half the
bytes, and they are widened to bf16 where the experts are:

    recv = widen(dispatch(rows of 8 bits, ids))

and back: the gradients for x, the gate weights and both weights.  Everything is
stream-ordered with counts that only the device knows; buffers are allocated
once, and a call may be captured into a CUDA graph (after one call of its kind).
"""
from __future__ import annotations

import torch

from . import hoc


class ExpertLayer:
    """Buffers of k ranks x `tokens` tokens of `hidden`, top-`topk` of `experts` experts of width `ffn`.

    capacity: rows of each rank's receive buffer.  The default, k * tokens * topk, has room for every pair at any
    rank; k * tokens * min(topk, experts / k) is enough where a token's experts are distinct.  A pair whose row does
    not fit is dropped, and status bit 0 says so.  wire8: forward takes x in rows of 8 bits."""

    def __init__(self, k: int, tokens: int, topk: int, hidden: int, ffn: int, experts: int, capacity: int | None = None,
                 device: int = 0, wire8: bool = False):
        if experts % k:
            raise ValueError("experts must be a multiple of the rank count")
        self.k, self.tokens, self.topk, self.hidden, self.ffn, self.experts = k, tokens, topk, hidden, ffn, experts
        self.per_rank = experts // k
        self.rows = k * tokens * topk if capacity is None else int(capacity)
        dev = torch.device("cuda", device)

        def ranks(*shape, dtype=torch.bfloat16):
            return [torch.empty(shape, dtype=dtype, device=dev) for _ in range(k)]

        self.recv, self.out = ranks(self.rows, hidden), ranks(self.rows, hidden)
        self.pre, self.h = ranks(self.rows, 2 * ffn), ranks(self.rows, ffn)
        self.dout, self.drecv, self.dpre = ranks(self.rows, hidden), ranks(self.rows, hidden), ranks(self.rows, 2 * ffn)
        self.pos = ranks(tokens * topk, dtype=torch.int32)
        self.counts = torch.empty((k, k), dtype=torch.int64, device=dev)
        self.seg = torch.empty((k, experts + 1), dtype=torch.int64, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.ones = [torch.ones(tokens * topk, device=dev)] * k
        self.ws = torch.empty(max(1, k * hoc.ep_pack_workspace(tokens, topk, experts)), dtype=torch.int32, device=dev)
        self.caps = [self.rows * hidden] * k
        self.recv8 = None
        if wire8:
            n = hoc.wire8_bytes(hidden)
            self.recv8 = ranks(self.rows, n, dtype=torch.uint8)
            self.caps8 = [self.rows * (n // 2)] * k
        torch.cuda.current_stream(dev).synchronize()  # status and ones are there for calls on any stream

    def forward(self, x, ids, gate, w_up, w_down, y, stream=None):
        """y[s] [tokens, hidden] of every source s; x[s] [tokens, hidden] bf16, or uint8 [tokens, wire8_bytes(hidden)] rows
        of 8 bits with wire8; ids[s] [tokens * topk] int32, gate[s] [tokens * topk] float32."""
        if self.recv8 is None:
            hoc.ep_dispatch_fused(ids, x, self.experts, self.recv, self.caps, self.pos, self.counts, self.ws, self.status,
                                  stream=stream)
            hoc.ep_segments(ids, self.experts, self.topk, self.seg, stream=stream)
        else:
            if any(v.dtype is not torch.uint8 or v.shape != (self.tokens, self.recv8[0].shape[1]) for v in x):
                raise ValueError(f"x: expected rows of 8 bits, uint8 [{self.tokens}, {self.recv8[0].shape[1]}]")
            hoc.ep_dispatch_fused(ids, [v.view(torch.bfloat16) for v in x], self.experts, self.recv8, self.caps8, self.pos,
                                  self.counts, self.ws, self.status, stream=stream)
            hoc.ep_segments(ids, self.experts, self.topk, self.seg, stream=stream)
            hoc.expert_widen(self.recv8, self.seg, self.recv, counts=self.counts, stream=stream)
        hoc.expert_mm(self.recv, w_up, self.seg, self.h, status=self.status, act="swiglu", pre=self.pre, stream=stream)
        hoc.expert_mm(self.h, w_down, self.seg, self.out, status=self.status, stream=stream)
        hoc.ep_combine_fused(self.out, self.caps, ids, self.pos, self.counts, gate, self.tokens, self.topk, self.hidden,
                             self.experts, y, self.status, stream=stream)

    def backward(self, dy, ids, gate, w_up, w_down, dx, dgate, dw_up, dw_down, accumulate: bool = False, stream=None):
        """Gradients of the last forward: dx[s] and dgate[s] of every source, dw_up[d] and dw_down[d] (bf16 or
        float32; added to with accumulate) of every rank."""
        st = self.status
        hoc.ep_combine_grad(dy, self.out, self.caps, ids, self.pos, self.counts, gate, self.tokens, self.topk,
                            self.hidden, self.experts, self.dout, dgate, st, stream=stream)
        hoc.expert_mm_wgrad(self.dout, self.h, self.seg, dw_down, status=st, accumulate=accumulate, stream=stream)
        hoc.expert_mm_dgrad(self.dout, w_down, self.seg, self.dpre, status=st, act="swiglu", pre=self.pre, stream=stream)
        hoc.expert_mm_wgrad(self.dpre, self.recv, self.seg, dw_up, status=st, accumulate=accumulate, stream=stream)
        hoc.expert_mm_dgrad(self.dpre, w_up, self.seg, self.drecv, status=st, stream=stream)
        hoc.ep_combine_fused(self.drecv, self.caps, ids, self.pos, self.counts, self.ones, self.tokens, self.topk,
                             self.hidden, self.experts, dx, st, stream=stream)
