"""Mx4Experts: the experts' gated MLP in microscaled 4-bit floating point, between a router's align and combine.

    hidden --moe_gather_mx4--> expert-grouped rows --moe_grouped_gemm_mx4, gate--> bf16 rows
           --moe_quantize_mx4--> 4-bit rows --moe_grouped_gemm_mx4--> expert outputs, for moe_combine

The weights are quantised once, at construction; every buffer is preallocated for the router's sizes, so that a step
(``MoeRouter.step_mx4``) neither allocates nor synchronises and can be captured in a CUDA graph.  Steps that may run at
the same time (on two streams, or two captured graphs) need objects, and routers, of their own.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import binding as B


class Mx4Experts:
    """w_up [E_local, 2 I, H] bf16 (the gate's I features, then the others), w_down [E_local, H, I] bf16."""

    def __init__(self, w_up: torch.Tensor, w_down: torch.Tensor, capacity: int):
        if w_up.dim() != 3 or w_down.dim() != 3:
            raise ValueError("w_up must be [E_local, 2 I, H], w_down [E_local, H, I]")
        E, two_i, H = w_up.shape
        if two_i % 2 != 0 or tuple(w_down.shape) != (E, H, two_i // 2):
            raise ValueError(f"w_down must be [{E}, {H}, {two_i // 2}] for w_up {tuple(w_up.shape)}, "
                             f"got {tuple(w_down.shape)}")
        self.E_local, self.H, self.I, self.capacity = E, H, two_i // 2, capacity
        dev = w_up.device
        self.w_up = B.moe_quantize_mx4(w_up.reshape(E * two_i, H))
        self.w_down = B.moe_quantize_mx4(w_down.reshape(E * H, self.I))
        self.rows = B.alloc_mx4(capacity, H, dev)
        self.act = torch.empty((capacity, self.I), dtype=torch.bfloat16, device=dev)
        self.act_rows = B.alloc_mx4(capacity, self.I, dev)
        self.out = torch.empty((capacity, H), dtype=torch.bfloat16, device=dev)

    def forward(self, hidden: torch.Tensor, k: int, align: B.AlignResult,
                device_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """The experts' outputs [capacity, H] for the routes of `align` (this object's buffer)."""
        if align.capacity != self.capacity or align.counts.numel() != self.E_local:
            raise ValueError(f"the layout has {align.capacity} rows of {align.counts.numel()} experts, this object "
                             f"{self.capacity} of {self.E_local}")
        B.moe_gather_mx4(hidden, k, align.inv_perm, self.capacity, self.rows, device_status, stream)
        B.moe_grouped_gemm_mx4(self.rows, self.w_up, align.counts, align.offsets, self.act, True, device_status, stream)
        B.moe_quantize_mx4(self.act, self.act_rows, align.num_tokens_post_pad, stream)
        return B.moe_grouped_gemm_mx4(self.act_rows, self.w_down, align.counts, align.offsets, self.out, False,
                                      device_status, stream)
