"""Trains the second projection of a small expert layer, then serves the layer in 4 bits.

Training: y = moe_grouped_gemm(act, w2), a squared error against a target, gradients from
moe_grouped_gemm_backward, a few steps of gradient descent on w2. Serving: the layer's weights
are quantised (moe_mxfp4_quantize) and a batch and a single token go through Mxfp4Experts, beside
the bf16 layer (moe_layer_forward). Needs one GB300.

    python examples/train_and_serve_mxfp4.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import mixture_experts_routing_token_gb300 as moe
from mixture_experts_routing_token_gb300.mxfp4_layer import Mxfp4Experts


def main(T=512, H=256, I=384, E=8, k=2, steps=20, rate=0.08, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s, scale=1.0: (torch.randn(*s, device="cuda", generator=gen) * scale).bfloat16()  # noqa: E731
    hidden, logits = normal(T, H), torch.randn(T, E, device="cuda", generator=gen)
    w13, w2, target = normal(E, 2 * I, H, scale=H ** -0.5), normal(E, H, I, scale=I ** -0.5), normal(E, H, I, scale=I ** -0.5)

    weights, indices = moe.moe_gating_softmax_topk(logits, k)
    r = moe.moe_align_by_expert(indices, weights, E)
    x = moe.moe_gather_rows(hidden, r["sorted_token_ids"], r["offsets"], k)
    gate, up = moe.moe_grouped_gemm(x, w13, r["offsets"]).float().chunk(2, dim=1)
    act = (torch.nn.functional.silu(gate) * up).bfloat16()
    want = moe.moe_grouped_gemm(act, target, r["offsets"]).float()
    # one learning rate per expert: a mean over its rows, against the activations' mean square; with n rows
    # of I features the largest curvature is about (1 + sqrt(I / n))^2, 12 here, so the rate stays below 2 / 12
    counts = r["counts"].clamp(min=1).float()
    step = (rate / counts / act.float().square().mean())[:, None, None]
    master, losses = w2.float(), []
    for _ in range(steps):
        err = moe.moe_grouped_gemm(act, w2, r["offsets"]).float() - want
        losses.append(float(err.square().mean()))
        _, d_w2 = moe.moe_grouped_gemm_backward(act, w2, r["offsets"], err.bfloat16(), want_d_x=False)
        master -= step * d_w2.float()
        w2 = master.bfloat16()
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps")

    experts = Mxfp4Experts(w13, w2)
    errors = []
    for n in (T, 1):
        full = moe.moe_layer_forward(hidden[:n].contiguous(), logits[:n].contiguous(), w13, w2, k).float()
        small = experts(hidden[:n].contiguous(), logits[:n].contiguous(), k).float()
        errors.append(float((small - full).norm() / full.norm()))
        print(f"{n} tokens: 4-bit layer against bf16, relative error {errors[-1]:.3f}")
    return losses, errors


if __name__ == "__main__":
    main()
