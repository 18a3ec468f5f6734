"""One training step of the top-k block through the C ABI (include/moe_topk.h).

MoETopKGate owns the device buffers (allocated with torch: plumbing only) and runs,
in stream order,

    moe_layer_norm_fwd -> moe_topk_route -> moe_topk_fwd            (forward)
    moe_topk_bwd -> moe_topk_route_bwd -> moe_layer_norm_bwd        (backward)

It is MoETop1Gate's sibling for K experts per token in 16-bit types: the block's input
x [T, H] is normalised (optional), the caller's gate logits [T, E] choose K experts per
token with weights, y [T, H] is the weighted sum of their linears, and the backward
gives the gradients of x, of the gate logits (through the weights), of the experts and
of the norm's parameters. The balance bias, if any, is the caller's to update between
steps (in place): it takes part in the choice only. Nothing here allocates or
synchronises after construction, so a step can be captured in a CUDA graph.
"""
from __future__ import annotations

import torch

from . import ops


class MoETopKGate:
    def __init__(self, W: torch.Tensor, bias: torch.Tensor | None, T: int, rule: ops.TopKRule,
                 gamma: torch.Tensor | None = None, beta: torch.Tensor | None = None, norm: bool = True,
                 eps: float = 1e-5, balance_bias: torch.Tensor | None = None,
                 logits_dtype: torch.dtype = torch.float32):
        """W [E, H, H] and bias [E, H] (or None) bfloat16 or float16 on the current device; gamma and
        beta [H] of the same type or float32. norm = False leaves the layer norm out."""
        E, H = W.shape[0], W.shape[1]
        if E != rule.E:
            raise ValueError(f"W: expected {rule.E} experts, got {E}")
        if not norm and (gamma is not None or beta is not None):
            raise ValueError("gamma and beta belong to the layer norm")
        dev, dt, f32 = W.device, W.dtype, torch.float32
        self.W, self.bias, self.T, self.E, self.H, self.rule = W, bias, T, E, H, rule
        self.gamma, self.beta, self.norm, self.eps, self.balance_bias = gamma, beta, norm, eps, balance_bias
        K = rule.K
        new = lambda *s, dtype=dt: torch.empty(*s, dtype=dtype, device=dev)  # noqa: E731
        self.routing = ops.Routing.empty(T * K, E, dev)
        self.weights, self.d_weights = new(T, K, dtype=f32), new(T, K, dtype=f32)
        self.y, self.d_normed = new(T, H), new(T, H)
        self.dW = torch.empty_like(W)
        self.db = None if bias is None else torch.empty_like(bias)
        self.d_logits = new(T, E, dtype=logits_dtype)
        if norm:
            self.normed, self.d_x = new(T, H), new(T, H)
            self.mean, self.rstd = new(T, dtype=f32), new(T, dtype=f32)
            self.dgamma = None if gamma is None else torch.empty_like(gamma)
            self.dbeta = None if beta is None else torch.empty_like(beta)
            self.norm_ws = ops.new_layer_norm_workspace(T, H, dev)
        else:
            self.d_x = self.d_normed
        self.ws = ops.new_topk_workspace(T, E, K, H, dev)

    def forward(self, x: torch.Tensor, gate_logits: torch.Tensor, stream=None) -> torch.Tensor:
        """y [T, H] (the gate's own buffer) of x [T, H] and gate_logits [T, E]."""
        if self.norm:
            ops.moe_layer_norm_fwd(x, self.gamma, self.beta, self.eps, self.normed, self.mean, self.rstd, stream)
        ops.moe_topk_route(gate_logits, self.rule, self.balance_bias, self.routing, self.weights, self.ws, stream)
        ops.moe_topk_fwd(self.normed if self.norm else x, self.W, self.bias, self.routing, self.weights, self.y, self.ws,
                         stream)
        return self.y

    def backward(self, x: torch.Tensor, gate_logits: torch.Tensor, d_y: torch.Tensor, accumulate_logits: bool = False,
                 stream=None):
        """After forward with the same x and gate_logits: d_x, d_logits, dW, db, dgamma and dbeta from
        d_y [T, H]. accumulate_logits adds to what self.d_logits holds (a balance loss's gradient that
        was written there, say; nothing is there before the first call)."""
        ops.moe_topk_bwd(self.normed if self.norm else x, self.W, self.bias, d_y, self.routing, self.weights,
                         self.d_normed, self.dW, self.db, self.d_weights, self.ws, stream)
        ops.moe_topk_route_bwd(gate_logits, self.rule, self.routing.expert_idx, self.d_weights, self.d_logits,
                               accumulate_logits, stream)
        if self.norm:
            ops.moe_layer_norm_bwd(x, self.d_normed, self.gamma, self.mean, self.rstd, self.d_x, self.dgamma, self.dbeta,
                                   self.norm_ws, stream)

    def step(self, x: torch.Tensor, gate_logits: torch.Tensor, d_y: torch.Tensor, stream=None):
        self.forward(x, gate_logits, stream)
        self.backward(x, gate_logits, d_y, stream=stream)
