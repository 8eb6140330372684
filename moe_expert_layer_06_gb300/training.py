"""The MoE layer for training: forward, and the gradients of its input and of every weight.

    routing   moe_route_scored                     gradient: moe_route_scored_backward
    dispatch  moe_dispatch, the rows kept in 8 bits (moe_checkpoint_rows)
    experts   moe_expert_project (gate and up),    moe_expert_project_backward,
              moe_swiglu_checkpoint,               moe_swiglu_backward,
              moe_expert_project (down)            moe_expert_project_backward
    shared    the same as one expert of all tokens, as wide as the shared experts together
    combine   moe_combine                          moe_combine_backward

Between the passes `Buffers` keeps, for each of a token's k rows, the dispatched row and gate and up in
8 bits (with a power of two for each 128 columns) and the expert's output in bf16; for each token the
shared gate and up in 8 bits; and the routing.  h is computed again from what was kept.  With
keep_rows=False the dispatched rows are not kept but gathered again from x, which layer_backward takes
anyway: k * hidden bytes a token less between the passes, for a scratch of twice as many, and the gate's and up's
gradients are of the rows themselves instead of rows rounded to 8 bits.  The other
buffers are scratch, which layers may share.  A pass runs on one stream, the current one or `stream`,
without host synchronisation, and may be captured in a CUDA graph.  Buffers may be made on another
stream than the passes run on (they are ready when they are made); who changes the stream between a
layer's passes orders the two, and who drops Buffers waits for the passes or records the stream, as for
any tensor.

The products are of bf16 operands with fp32 sums; the gradient of the logits is rounded to bf16 once
for the router's products.  The routing's selection has no gradient, nor has select_bias.
"""
from __future__ import annotations

import contextlib

import torch

from . import (MOE_PAYLOAD_BLOCK, Project, Shape, moe_checkpoint_rows, moe_combine, moe_combine_backward, moe_dispatch,
               moe_dispatch_workspace_size, moe_expert_project, moe_expert_project_backward, moe_gather_rows,
               moe_route_scored, moe_route_scored_backward, moe_route_workspace_size, moe_swiglu_backward,
               moe_swiglu_checkpoint)


def _blocks(cols: int) -> int:
    return -(-cols // MOE_PAYLOAD_BLOCK)


def _on(stream):
    """The context in which torch's own operations run on `stream`."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream))


class Buffers:
    """What layer_forward leaves for layer_backward, and their scratch, for batches of T tokens.
    keep_rows: whether the dispatched rows are kept (in 8 bits), or gathered again from x."""

    def __init__(self, shape, T: int, device="cuda", keep_rows=True):
        s = Shape.of(shape)
        n, H, I, Is = T * s.top_k, s.hidden, s.inter, s.n_shared * s.inter_shared
        new = lambda dtype, *size: torch.empty(size, dtype=dtype, device=device)  # noqa: E731
        bf16, i32, f32, u8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
        self.T = T
        # kept
        self.logits, self.topk_idx, self.topk_w = new(f32, T, s.n_experts), new(i32, T, s.top_k), new(f32, T, s.top_k)
        self.slot_of, self.perm, self.inv_perm = (new(i32, n) for _ in range(3))
        self.counts, self.offsets, self.blocks = new(i32, s.n_slots + 1), new(i32, s.n_slots + 2), new(i32, s.n_blocks)
        self.x8, self.x8_scale = (new(u8, n, H), new(f32, n, _blocks(H))) if keep_rows else (None, None)
        self.act8, self.act8_scale = new(u8, n, 2 * I), new(f32, n, 2 * _blocks(I))
        self.y_disp = new(bf16, n, H)
        if Is:
            self.shared8, self.shared8_scale = new(u8, T, 2 * Is), new(f32, T, 2 * _blocks(Is))
        # scratch
        self.token_of, self.x_rows = (None, None) if keep_rows else (new(i32, n), new(bf16, n, H))
        self.rows = new(bf16, n, H)           # x_disp; dy_disp; dx_disp
        self.gate_up = new(bf16, n, 2 * I)    # and its gradient
        self.h, self.dh = new(bf16, n, I), new(bf16, n, I)
        self.x32 = new(f32, T, H)             # y_shared; what reaches dx beside the experts
        self.d_topk_w, self.d_logits = new(f32, T, s.top_k), new(f32, T, s.n_experts)
        self.d_logits16 = new(bf16, T, s.n_experts)
        if Is:
            self.shared_gate_up, self.shared_h, self.shared_dh = new(bf16, T, 2 * Is), new(bf16, T, Is), new(bf16, T, Is)
        self.ones = torch.ones((T, s.top_k), device=device)
        self.all_tokens = torch.tensor([0, T], dtype=i32, device=device)  # offsets of the one slot of dense products
        self.ws = new(u8, max(moe_route_workspace_size(s, T), moe_dispatch_workspace_size(s, T), 16))
        # ones and all_tokens are filled, and what held this memory before is over, whatever stream reads them first
        torch.cuda.current_stream(self.ws.device).synchronize()


def _check(s: Shape, buffers: Buffers, T: int):
    if buffers.T != T:
        raise ValueError(f"buffers are for {buffers.T} tokens, the batch has {T}")
    if s.n_slots != s.n_experts:
        raise ValueError("training takes a layer without replicas (n_slots = n_experts)")
    if s.n_experts % 8 or s.hidden % 16:
        raise ValueError("training needs n_experts in multiples of 8 and hidden in multiples of 16")


def layer_forward(shape, router, T: int, x, w_router, select_bias, w_gate, w_up, w_down, ws_gate, ws_up, w_shared_down, out,
                  buffers: Buffers, stream=None) -> Buffers:
    """out [T, H] bf16: the layer's output.  Weights as moe_forward's, but w_shared_down
    [H, n_sh*I_sh] (tenants.shared_down_matrix); the shared ones None without shared experts."""
    s, b = Shape.of(shape), buffers
    _check(s, b, T)
    n, H, I, Is = T * s.top_k, s.hidden, s.inter, s.n_shared * s.inter_shared
    moe_route_scored(s, router, T, x, w_router, select_bias, None, b.logits, b.topk_idx, b.topk_w, b.ws, stream=stream)
    moe_dispatch(s, T, x, b.topk_idx, None, b.slot_of, b.counts, b.blocks, b.offsets, b.perm, b.inv_perm, b.rows, b.ws,
                 stream=stream)
    if b.x8 is not None:
        moe_checkpoint_rows(n, H, b.rows, b.x8, b.x8_scale, stream=stream)
    moe_expert_project(Project(H, I, s.n_slots, 2), n, b.rows, b.offsets, w_gate, w_up, b.gate_up, stream=stream)
    moe_swiglu_checkpoint(n, I, b.gate_up, b.h, b.act8, b.act8_scale, stream=stream)
    moe_expert_project(Project(I, H, s.n_slots), n, b.h, b.offsets, w_down, None, b.y_disp, stream=stream)
    if Is:
        moe_expert_project(Project(H, Is, 1, 2), T, x, b.all_tokens, ws_gate.view(1, Is, H), ws_up.view(1, Is, H), b.shared_gate_up,
                           stream=stream)
        moe_swiglu_checkpoint(T, Is, b.shared_gate_up, b.shared_h, b.shared8, b.shared8_scale, stream=stream)
        moe_expert_project(Project(Is, H, 1), T, b.shared_h, b.all_tokens, w_shared_down.view(1, H, Is), None, b.x32, stream=stream)
    moe_combine(s, T, b.y_disp, b.inv_perm, b.topk_w, b.x32 if Is else None, out, stream=stream)
    return b


def layer_backward(shape, router, T: int, d_out, x, w_router, w_gate, w_up, w_down, ws_gate, ws_up, w_shared_down, dx, d_w_router,
                   d_w_gate, d_w_up, d_w_down, d_ws_gate, d_ws_up, d_w_shared_down, buffers: Buffers, add=False, stream=None):
    """Gradients of layer_forward's last call on these buffers, with the same x: dx [T, H] bf16, and every weight's as
    the weight (bf16 or fp32; with add, fp32 values that they are added to)."""
    s, b = Shape.of(shape), buffers
    _check(s, b, T)
    n, H, I, E, Is = T * s.top_k, s.hidden, s.inter, s.n_experts, s.n_shared * s.inter_shared
    down, gate_up, logits = Project(I, H, s.n_slots), Project(H, I, s.n_slots, 2), Project(H, E, 1)
    # combine, down, SwiGLU, gate and up
    moe_combine_backward(s, T, d_out, b.y_disp, b.inv_perm, b.topk_w, b.rows, b.d_topk_w, stream=stream)
    moe_expert_project_backward(down, n, b.rows, None, None, None, b.offsets, w_down, None, b.dh, None, stream=stream)
    moe_swiglu_backward(n, I, b.act8, b.act8_scale, b.dh, b.gate_up, b.h, stream=stream)
    moe_expert_project_backward(down, n, b.rows, b.h, None, None, b.offsets, None, None, None, d_w_down, add_dw=add, stream=stream)
    if b.x8 is None and n:
        with _on(stream):
            torch.floor_divide(b.perm, s.top_k, out=b.token_of)
        moe_gather_rows(x, b.token_of, b.x_rows, stream=stream)
    moe_expert_project_backward(gate_up, n, b.gate_up, b.x_rows, b.x8, b.x8_scale, b.offsets, w_gate, w_up, b.rows, d_w_gate, d_w_up,
                                add_dw=add, stream=stream)
    # router
    moe_route_scored_backward(s, router, T, b.logits, b.topk_idx, b.d_topk_w, b.d_logits, stream=stream)
    with _on(stream):
        b.d_logits16.copy_(b.d_logits)
    moe_expert_project_backward(logits, T, b.d_logits16, x, None, None, b.all_tokens, w_router.view(1, E, H), None, b.x32,
                                d_w_router.view(1, E, H), add_dw=add, stream=stream)
    # shared experts: their dx is added to the router's
    if Is:
        one = lambda t: t.view(1, Is, H)  # noqa: E731
        shared_down, shared = Project(Is, H, 1), Project(H, Is, 1, 2)
        moe_expert_project_backward(shared_down, T, d_out, None, None, None, b.all_tokens, w_shared_down.view(1, H, Is), None,
                                    b.shared_dh, None, stream=stream)
        moe_swiglu_backward(T, Is, b.shared8, b.shared8_scale, b.shared_dh, b.shared_gate_up, b.shared_h, stream=stream)
        moe_expert_project_backward(shared_down, T, d_out, b.shared_h, None, None, b.all_tokens, None, None, None,
                                    d_w_shared_down.view(1, H, Is), add_dw=add, stream=stream)
        moe_expert_project_backward(shared, T, b.shared_gate_up, x, None, None, b.all_tokens, one(ws_gate), one(ws_up), b.x32,
                                    one(d_ws_gate), one(d_ws_up), add_dx=True, add_dw=add, stream=stream)
    moe_combine(s, T, b.rows, b.inv_perm, b.ones, b.x32, dx, stream=stream)


__all__ = ["Buffers", "layer_backward", "layer_forward"]
