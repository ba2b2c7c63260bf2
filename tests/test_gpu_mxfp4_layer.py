"""The 4-bit expert layer: the composition of its calls bit for bit, close to the bf16 layer, on a
stream and in a graph; and the example that trains and serves."""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT
from gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu


def make(T, H, I, E, seed=0):
    g = torch.Generator().manual_seed(seed)
    normal = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).bfloat16().to(DEV)  # noqa: E731
    return (normal(T, H), torch.randn(T, E, generator=g).to(DEV), normal(E, 2 * I, H, scale=H ** -0.5),
            normal(E, H, I, scale=I ** -0.5))


@pytest.mark.parametrize("T,H,I,E,k", [(1, 128, 96, 8, 2), (5, 256, 160, 16, 4), (700, 256, 384, 8, 2), (300, 64, 32, 4, 4)])
def test_layer_is_its_calls(T, H, I, E, k):
    moe = need_gpu()
    from mixture_experts_routing_token_gb300.mxfp4_layer import Mxfp4Experts
    hidden, logits, w13, w2 = make(T, H, I, E)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = Mxfp4Experts(w13, w2)(hidden, logits, k, status=status)
    assert int(status.item()) == 0
    weights, indices = moe.moe_gating_softmax_topk(logits, k)
    r = moe.moe_align_by_expert(indices, weights, E)
    x = moe.moe_mxfp4_quantize(moe.moe_gather_rows(hidden, r["sorted_token_ids"], r["offsets"], k))
    act = moe.moe_mxfp4_grouped_gemm(*x, *moe.moe_mxfp4_quantize(w13), r["offsets"], activation="silu_and_mul")
    y = moe.moe_mxfp4_grouped_gemm(*moe.moe_mxfp4_quantize(act), *moe.moe_mxfp4_quantize(w2), r["offsets"])
    want = moe.moe_ep_combine(y, weights, r["reverse_indices"], r["offsets"])
    assert torch.equal(got, want)
    # a value of a normal block is off by about a tenth (a grid step is a quarter to a half of the value,
    # its rms error the step over sqrt(12)); four operands with such errors add up to about a quarter
    full = moe.moe_layer_forward(hidden, logits, w13, w2, k).float()
    assert float((got.float() - full).norm() / full.norm()) < 0.4


def test_layer_in_a_graph_on_a_stream():
    moe = need_gpu()
    from mixture_experts_routing_token_gb300.mxfp4_layer import Mxfp4Experts
    hidden, logits, w13, w2 = make(40, 128, 128, 8)
    layer = Mxfp4Experts(w13, w2)
    want = layer(hidden, logits, 2)
    h, lg, out = torch.zeros_like(hidden), logits.clone(), torch.empty_like(hidden)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(h, lg, 2, out=out)
    h.copy_(hidden)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_layer_without_tokens():
    moe = need_gpu()
    from mixture_experts_routing_token_gb300.mxfp4_layer import Mxfp4Experts
    hidden, logits, w13, w2 = make(1, 64, 64, 4)
    assert Mxfp4Experts(w13, w2)(hidden[:0], logits[:0], 2).shape == (0, 64)


def test_layer_refusals():
    need_gpu()
    from mixture_experts_routing_token_gb300.mxfp4_layer import Mxfp4Experts
    hidden, logits, w13, w2 = make(3, 64, 64, 4)
    with pytest.raises(ValueError, match="w13 must be"):
        Mxfp4Experts(w13, w2[:, :, :32].contiguous())
    with pytest.raises(ValueError, match="multiples of 32"):
        Mxfp4Experts(w13[:, :80].contiguous(), w2[:, :, :40].contiguous())
    with pytest.raises(ValueError, match="router_logits"):
        Mxfp4Experts(w13, w2)(hidden, logits[:, :2].contiguous(), 2)


def test_example_trains_and_serves():
    need_gpu()
    spec = importlib.util.spec_from_file_location("example", os.path.join(ROOT, "examples", "train_and_serve_mxfp4.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, errors = example.main(T=256, steps=8)
    assert losses[-1] < 0.7 * losses[0]
    assert max(errors) < 0.4
