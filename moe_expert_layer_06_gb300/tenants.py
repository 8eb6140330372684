"""The MoE layer for a batch of many tenants: scored routing, and each request's
low-rank adapter on the shared experts' down projection.

    routing   moe_route_scored (sigmoid or softmax scores, a balance bias, groups)
    dispatch  moe_dispatch
    experts   moe_expert_gate_up, then moe_expert_down for the routed experts
    shared    moe_adapter_project: one [H, n_sh*I_sh] matrix for all requests, and
              beside it the adapter of each token's request
    combine   moe_combine

Everything runs on one stream without host synchronisation; `Buffers` holds what
the steps pass on, so a serving loop allocates once and may capture the call in
a CUDA graph.
"""
from __future__ import annotations

import torch

from . import (MOE_FFN_AUTO, Adapter, Shape, moe_adapter_project, moe_adapter_workspace_size, moe_combine, moe_dispatch,
               moe_dispatch_workspace_size, moe_expert_down, moe_expert_gate_up, moe_route_scored,
               moe_route_workspace_size)


def shared_down_matrix(ws_down: torch.Tensor) -> torch.Tensor:
    """ws_down [n_sh, H, I_sh] as the one matrix [H, n_sh*I_sh] on the
    concatenated shared intermediate (the sum over the shared experts is then
    part of the contraction).  Done once, when the weights are loaded."""
    n, h, i = ws_down.shape
    return ws_down.permute(1, 0, 2).reshape(h, n * i).contiguous()


class Buffers:
    """Intermediates of tenant_forward for batches of T tokens."""

    def __init__(self, shape, adapter: Adapter, T: int, device="cuda"):
        s = Shape.of(shape)
        n, i32, bf16 = T * s.top_k, dict(dtype=torch.int32, device=device), dict(dtype=torch.bfloat16, device=device)
        self.T = T
        self.topk_idx = torch.empty((T, s.top_k), **i32)
        self.topk_w = torch.empty((T, s.top_k), device=device)
        self.slot_of, self.perm, self.inv_perm = (torch.empty(n, **i32) for _ in range(3))
        self.counts, self.offsets = torch.empty(s.n_slots + 1, **i32), torch.empty(s.n_slots + 2, **i32)
        self.blocks = torch.empty(s.n_blocks, **i32)
        self.x_disp, self.y_disp = torch.empty((n, s.hidden), **bf16), torch.empty((n, s.hidden), **bf16)
        self.h_disp = torch.empty((n, s.inter), **bf16)
        self.h_shared = torch.empty((T, s.n_shared * s.inter_shared), **bf16)
        self.y_shared = torch.empty((T, s.hidden), device=device)
        need = max(moe_route_workspace_size(s, T), moe_dispatch_workspace_size(s, T),
                   moe_adapter_workspace_size(adapter, T), 16)
        self.ws = torch.empty(need, dtype=torch.uint8, device=device)


def tenant_forward(shape, router, adapter: Adapter, T: int, x, w_router, select_bias, w_gate, w_up, w_down, ws_gate, ws_up,
                   w_shared_down, lora_a, lora_b, scaling, adapter_of, out, buffers: Buffers, replica_of=None,
                   mode: int = MOE_FFN_AUTO, stream=None) -> Buffers:
    """out [T, H] bf16: the layer's output for T tokens of requests with adapters
    adapter_of [T] (-1: none).  w_shared_down [H, n_sh*I_sh] (shared_down_matrix);
    lora_a [n, r, n_sh*I_sh], lora_b [n, H, r]; adapter = Adapter(n_sh*I_sh, H, n, r).
    Other weights as moe_forward's.  Returns the buffers (routing, counts)."""
    s = Shape.of(shape)
    if adapter.in_features != s.n_shared * s.inter_shared or adapter.out_features != s.hidden:
        raise ValueError("the adapter's features must be n_shared * inter_shared and hidden")
    if buffers.T != T:
        raise ValueError(f"buffers are for {buffers.T} tokens, the batch has {T}")
    b = buffers
    moe_route_scored(s, router, T, x, w_router, select_bias, None, None, b.topk_idx, b.topk_w, b.ws, stream=stream)
    moe_dispatch(s, T, x, b.topk_idx, replica_of, b.slot_of, b.counts, b.blocks, b.offsets, b.perm, b.inv_perm, b.x_disp,
                 b.ws, stream=stream)
    moe_expert_gate_up(s, T, x, b.x_disp, b.offsets, w_gate, w_up, ws_gate, ws_up, b.h_disp, b.h_shared, mode, stream=stream)
    routed = Shape(s.hidden, s.inter, s.n_experts, s.top_k, 0, 0, s.n_slots, s.n_blocks)
    moe_expert_down(routed, T, b.h_disp, None, b.offsets, w_down, None, b.y_disp, None, mode, stream=stream)
    moe_adapter_project(adapter, T, b.h_shared, w_shared_down, lora_a, lora_b, scaling, adapter_of, b.y_shared, None, b.ws,
                        stream=stream)
    moe_combine(s, T, b.y_disp, b.inv_perm, b.topk_w, b.y_shared, out, stream=stream)
    return b


__all__ = ["Buffers", "shared_down_matrix", "tenant_forward"]
