"""An expert layer with what stands around it, over simulated ranks on one GPU, forward and backward.

HOCCL section 2.1: token dispatch and combine surround the experts of a layer.  This driver runs the block of a model that
such a layer is a part of, from the residual stream and back to it (include/hoc_block.h, expert_layer.py):

    h     = x + residual                          the residual stream
    n     = rms_norm(h) * norm                    and in rows of 8 bits for the dispatch, if asked for
    ids, gate = route(n router^T)                 topk of the experts, by softmax or sigmoid scores
    y     = h + dropout(experts(n, ids, gate))

and the gradients for x (and the residual), the norm's weight, the router and the experts' weights.  The tokens of all
ranks lie in one buffer, rank by rank.  Everything is stream-ordered with counts that only the device knows; buffers are
allocated once, and a call may be captured into a CUDA graph (after one call of its kind).
"""
from __future__ import annotations

import torch

from . import hoc
from .expert_layer import ExpertLayer


class ExpertBlock:
    """Buffers of k ranks x `tokens` tokens of `hidden`, top-`topk` of `experts` experts of width `ffn`.

    score, groups, top_groups, renormalise and scale are the routing's (hoc.ep_route), whose logits and their gradients are
    stored in bf16, as hoc.linear writes them; drop the probability of the dropout; wire8: tokens go to their experts in rows
    of 8 bits; capacity: as ExpertLayer's."""

    def __init__(self, k: int, tokens: int, topk: int, hidden: int, ffn: int, experts: int, *, score: str = "softmax",
                 groups: int = 1, top_groups: int | None = None, renormalise: bool = True, scale: float = 1.0,
                 eps: float = 1e-6, drop: float = 0.0, wire8: bool = False, capacity: int | None = None, device: int = 0):
        self.layer = ExpertLayer(k, tokens, topk, hidden, ffn, experts, capacity, device, wire8)
        self.k, self.tokens, self.eps, self.drop = k, tokens, eps, drop
        self.routing = dict(score=score, renormalise=renormalise, scale=scale)
        self.choice = dict(groups=groups, top_groups=top_groups)
        dev, n = torch.device("cuda", device), k * tokens

        def rows(width, dtype=torch.bfloat16):
            return torch.empty((n, width), dtype=dtype, device=dev)

        self.h, self.n, self.out = rows(hidden), rows(hidden), rows(hidden)
        self.wire = rows(hoc.wire8_bytes(hidden), torch.uint8) if wire8 else None
        self.logits, self.dlogits = rows(experts), rows(experts)
        self.dout, self.dn, self.dn_router = rows(hidden), rows(hidden), rows(hidden)
        self.ids = torch.empty(n * topk, dtype=torch.int32, device=dev)
        self.gate, self.dgate = (torch.empty(n * topk, device=dev) for _ in range(2))
        self.ws = torch.empty(hoc.rms_norm_workspace(n, hidden), dtype=torch.int32, device=dev)
        self.no_seed = torch.zeros(2, dtype=torch.int64, device=dev)
        self.status = self.layer.status
        self.held = None
        torch.cuda.current_stream(dev).synchronize()  # no_seed is there for calls on any stream

    def _ranks(self, t):
        return list(t.chunk(self.k)) if t.shape[0] else [t] * self.k

    def forward(self, x, norm, router, w_up, w_down, y, *, residual=None, bias=None, seed=None, stream=None):
        """y [k * tokens, hidden] = the residual stream behind the block; x and residual as y; norm [hidden]; router [experts,
        hidden]; w_up[d], w_down[d] as ExpertLayer's; bias float32 [experts] for the choice; seed: two int64 for the
        dropout, if there is one.  Keeps what the backward pass needs; x itself where there is no residual, which has to stay
        as it is until then: y may be x, or the residual, but without a residual a y that is x leaves no backward pass."""
        if self.drop and seed is None:
            raise ValueError("seed: the dropout needs one")
        held, self.held = self.h if residual is not None else x, None  # (until the whole pass is queued)
        hoc.rms_norm(x, norm, self.n, eps=self.eps, residual=residual, h=self.h if residual is not None else None,
                     wire=self.wire, stream=stream)
        hoc.linear(self.n, router, self.logits, status=self.status, stream=stream)
        hoc.ep_route(self.logits, self.ids, self.gate, bias=bias, **self.routing, **self.choice, stream=stream)
        self.layer.forward(self._ranks(self.n if self.wire is None else self.wire), self._ranks(self.ids),
                           self._ranks(self.gate), w_up, w_down, self._ranks(self.out), stream=stream)
        hoc.dropout(self.out, y, self.drop, self.no_seed if seed is None else seed, residual=held, stream=stream)
        if residual is not None or y.data_ptr() != x.data_ptr() or not x.numel():  # else what backward would read is gone
            self.held = held

    def backward(self, dy, norm, router, w_up, w_down, dx, dnorm, drouter, dw_up, dw_down, *, seed=None,
                 accumulate: bool = False, stream=None):
        """Gradients of the last forward, which had these weights and this seed: dx [k * tokens, hidden] for x and for the
        residual alike; dnorm, drouter, dw_up[d] and dw_down[d] in bf16 or float32 (added to with accumulate)."""
        if self.held is None:
            raise ValueError("no forward pass to go back through: there was none, or it wrote y over the x that is needed here")
        dout = dy
        if self.drop:
            if seed is None:
                raise ValueError("seed: the dropout needs one")
            dout = self.dout
            hoc.dropout(dy, dout, self.drop, seed, stream=stream)
        self.layer.backward(self._ranks(dout), self._ranks(self.ids), self._ranks(self.gate), w_up, w_down,
                            self._ranks(self.dn), self._ranks(self.dgate), dw_up, dw_down, accumulate, stream=stream)
        hoc.ep_route_grad(self.logits, self.ids, self.dgate, self.dlogits, **self.routing, stream=stream)
        hoc.linear_wgrad(self.dlogits, self.n, drouter, status=self.status, accumulate=accumulate, stream=stream)
        hoc.linear_dgrad(self.dlogits, router, self.dn_router, status=self.status, stream=stream)
        hoc.rms_norm_grad(self.dn, self.held, norm, dx, eps=self.eps, dy2=self.dn_router, dres=dy, dw=dnorm,
                          accumulate=accumulate, workspace=self.ws, stream=stream)
