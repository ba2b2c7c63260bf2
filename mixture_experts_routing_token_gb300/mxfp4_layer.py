"""MoE layer whose experts hold 4-bit microscaled weights (serving).

The weights are quantised once, to 4.25 bits a value; a
forward pass quantises the activations in front of each product:

1. ``moe_gating_softmax_topk`` and ``moe_align_by_expert``;
2. ``moe_mxfp4_quantize`` with ``rows=sorted_token_ids``: the token rows, quantised and
   brought into expert order in one step;
3. ``moe_mxfp4_grouped_gemm`` with w13 and ``activation="silu_and_mul"`` -> bf16 activations;
4. ``moe_mxfp4_quantize`` of those, ``moe_mxfp4_grouped_gemm`` with w2;
5. ``moe_ep_combine``: out[t] = sum_j w[t, j] y[pos(t, j)].

Everything runs on the caller's stream without host synchronisation, so a step can be captured
into a CUDA graph.
"""
from __future__ import annotations

import torch

from . import _binding as moe


class Mxfp4Experts:
    """w13 [E, 2I, H] and w2 [E, H, I] (float32, bf16 or float16 device tensors), held in 4 bits.

    H and I must be multiples of 32."""

    def __init__(self, w13: torch.Tensor, w2: torch.Tensor, stream=None):
        if w13.dim() != 3 or w2.dim() != 3 or w13.shape[1] % 2:
            raise ValueError("w13 must be [E, 2I, H] and w2 [E, H, I]")
        E, I2, H = w13.shape
        I = I2 // 2
        if tuple(w2.shape) != (E, H, I):
            raise ValueError("w13 must be [E, 2I, H] and w2 [E, H, I]")
        if H % 32 or I % 32:
            raise ValueError(f"H and I must be multiples of 32 (got H={H}, I={I})")
        self.E, self.H, self.I = E, H, I
        self.w13 = moe.moe_mxfp4_quantize(w13, stream=stream)
        self.w2 = moe.moe_mxfp4_quantize(w2, stream=stream)

    def forward(self, hidden, router_logits, k, norm_topk_prob=True, out=None, status=None, stream=None):
        """hidden [T, H] bf16, router_logits [T, E] float32 -> [T, H] bf16."""
        if hidden.dim() != 2 or hidden.shape[1] != self.H or tuple(router_logits.shape) != (hidden.shape[0], self.E):
            raise ValueError(f"hidden must be [T, {self.H}] and router_logits [T, {self.E}]")
        weights, indices = moe.moe_gating_softmax_topk(router_logits, k, norm_topk_prob, stream=stream)
        r = moe.moe_align_by_expert(indices, weights, self.E, status=status, stream=stream)
        x, xs = moe.moe_mxfp4_quantize(hidden, rows=r["sorted_token_ids"], status=status, stream=stream)
        act = moe.moe_mxfp4_grouped_gemm(x, xs, *self.w13, r["offsets"], activation="silu_and_mul", status=status,
                                         stream=stream)
        a, s = moe.moe_mxfp4_quantize(act, stream=stream)
        y = moe.moe_mxfp4_grouped_gemm(a, s, *self.w2, r["offsets"], status=status, stream=stream)
        return moe.moe_ep_combine(y, weights, r["reverse_indices"], r["offsets"], out=out, stream=stream)

    __call__ = forward
