"""MoE layer whose experts hold 8-bit weights with a scale for each 128 x 128 block (serving).

A forward pass runs on 8-bit rows with a scale for each 128 values:

1. ``moe_gating_softmax_topk`` and ``moe_align_by_expert``;
2. the token rows in 8 bits: ``moe_fp8_quantize``, or ``moe_rms_norm_fp8`` where the layer holds the norm in
   front of it (:meth:`Fp8Experts.block`); ``moe_fp8_gather_rows`` brings them into expert order;
3. ``moe_fp8_grouped_gemm`` with w13 and ``activation="silu_and_mul"`` -> bf16 activations;
4. ``moe_fp8_quantize`` of those, ``moe_fp8_grouped_gemm`` with w2;
5. ``moe_ep_combine``: out[t] = sum_j w[t, j] y[pos(t, j)].

Everything runs on the caller's stream without host synchronisation, so a step can be captured
into a CUDA graph.
"""
from __future__ import annotations

import contextlib

import torch

from . import _binding as moe


def _under(stream):
    """The caller's stream as the current one."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)))
    return torch.cuda.stream(stream)


class Fp8Experts:
    """w13 [E, 2I, H] and w2 [E, H, I] (float32, bf16 or float16 device tensors), held in 8 bits.

    H and I must be multiples of 16. ``norm`` [H] (bf16) is the weight of the root-mean-square norm that
    :meth:`block` applies first, ``eps`` its addend."""

    def __init__(self, w13: torch.Tensor, w2: torch.Tensor, norm: torch.Tensor | None = None, eps: float = 1e-6, stream=None):
        if w13.dim() != 3 or w2.dim() != 3 or w13.shape[1] % 2:
            raise ValueError("w13 must be [E, 2I, H] and w2 [E, H, I]")
        E, I2, H = w13.shape
        I = I2 // 2
        if tuple(w2.shape) != (E, H, I):
            raise ValueError("w13 must be [E, 2I, H] and w2 [E, H, I]")
        if H % 16 or I % 16:
            raise ValueError(f"H and I must be multiples of 16 (got H={H}, I={I})")
        if norm is not None and (tuple(norm.shape) != (H,) or norm.dtype != torch.bfloat16):
            raise ValueError(f"norm must be [{H}] bf16")
        self.E, self.H, self.I = E, H, I
        self.norm, self.eps = norm, eps
        self.w13 = moe.moe_fp8_quantize(w13, block_rows=moe.FP8_BLOCK, stream=stream)
        self.w2 = moe.moe_fp8_quantize(w2, block_rows=moe.FP8_BLOCK, stream=stream)

    def _experts(self, codes, scales, router_logits, k, norm_topk_prob, out, status, stream):
        weights, indices = moe.moe_gating_softmax_topk(router_logits, k, norm_topk_prob, stream=stream)
        r = moe.moe_align_by_expert(indices, weights, self.E, status=status, stream=stream)
        x, xs = moe.moe_fp8_gather_rows(codes, scales, r["sorted_token_ids"], r["offsets"], status=status, stream=stream)
        act = moe.moe_fp8_grouped_gemm(x, xs, *self.w13, r["offsets"], activation="silu_and_mul", status=status, stream=stream)
        a, s = moe.moe_fp8_quantize(act, stream=stream)
        y = moe.moe_fp8_grouped_gemm(a, s, *self.w2, r["offsets"], status=status, stream=stream)
        return moe.moe_ep_combine(y, weights, r["reverse_indices"], r["offsets"], out=out, stream=stream)

    def forward(self, hidden, router_logits, k, norm_topk_prob=True, out=None, status=None, stream=None):
        """hidden [T, H] bf16, router_logits [T, E] float32 -> [T, H] bf16."""
        if hidden.dim() != 2 or hidden.shape[1] != self.H or tuple(router_logits.shape) != (hidden.shape[0], self.E):
            raise ValueError(f"hidden must be [T, {self.H}] and router_logits [T, {self.E}]")
        codes, scales = moe.moe_fp8_quantize(hidden, stream=stream)
        return self._experts(codes, scales, router_logits, k, norm_topk_prob, out, status, stream)

    __call__ = forward

    def block(self, x, residual, router, k, norm_topk_prob=True, residual_out=None, out=None, status=None, stream=None):
        """The layer with the norm in front: h = x + residual, experts on norm(h) -> (out [T, H], h [T, H]).

        x, residual [T, H] bf16; ``router(n)`` maps the normed rows n [T, H] bf16 to float32 logits [T, E] (a product with
        the router's weights; the call's stream is the current one for it). The caller adds out to h, e.g. as the next block's x and residual."""
        if self.norm is None:
            raise ValueError("block needs the norm's weight: Fp8Experts(w13, w2, norm)")
        if x.dim() != 2 or x.shape[1] != self.H or x.dtype != torch.bfloat16 or tuple(residual.shape) != tuple(x.shape):
            raise ValueError(f"x must be [T, {self.H}] bf16 and residual as x")
        codes, scales, h, n = moe.moe_rms_norm_fp8(x, self.norm, residual=residual, eps=self.eps, want_normed=True,
                                                   residual_out=residual_out, stream=stream)
        with _under(stream):
            logits = router(n)
        if tuple(logits.shape) != (x.shape[0], self.E):
            raise ValueError(f"router must return [T, {self.E}]")
        return self._experts(codes, scales, logits, k, norm_topk_prob, out, status, stream), h
