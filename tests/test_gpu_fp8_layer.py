"""The 8-bit expert layer: the composition of its calls bit for bit, close to the bf16 layer, with the norm in front, on
another stream, in a graph; and a training step made of the sorted rows' calls and the grouped product's."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, need_gpu
from oracle import grouped, sorted_rows

pytestmark = pytest.mark.gpu


def make(T, H, I, E, seed=0):
    g = torch.Generator().manual_seed(seed)
    normal = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).bfloat16().to(DEV)  # noqa: E731
    return (normal(T, H), torch.randn(T, E, generator=g).to(DEV), normal(E, 2 * I, H, scale=H ** -0.5),
            normal(E, H, I, scale=I ** -0.5))


SIZES = [(1, 128, 96, 8, 2), (5, 256, 160, 16, 4), (700, 272, 400, 8, 2), (300, 64, 32, 4, 4)]


@pytest.mark.parametrize("T,H,I,E,k", SIZES)
def test_layer_is_its_calls(T, H, I, E, k):
    moe = need_gpu()
    from mixture_experts_routing_token_gb300.fp8_layer import Fp8Experts
    hidden, logits, w13, w2 = make(T, H, I, E)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = Fp8Experts(w13, w2)(hidden, logits, k, status=status)
    assert int(status.item()) == 0
    weights, indices = moe.moe_gating_softmax_topk(logits, k)
    r = moe.moe_align_by_expert(indices, weights, E)
    # rows sorted first, then quantised: the same rows
    x = moe.moe_fp8_quantize(moe.moe_gather_rows(hidden, r["sorted_token_ids"], r["offsets"], k))
    act = moe.moe_fp8_grouped_gemm(*x, *moe.moe_fp8_quantize(w13, block_rows=128), r["offsets"], activation="silu_and_mul")
    y = moe.moe_fp8_grouped_gemm(*moe.moe_fp8_quantize(act), *moe.moe_fp8_quantize(w2, block_rows=128), r["offsets"])
    assert torch.equal(got, moe.moe_ep_combine(y, weights, r["reverse_indices"], r["offsets"]))
    # a value is off by up to 2^-4 of itself, 0.6 of that over sqrt(3) rms (values spread over a binade): about 0.026;
    # four operands of two products: about 0.06 with the gate's product
    full = moe.moe_layer_forward(hidden, logits, w13, w2, k).float()
    assert float((got.float() - full).norm() / full.norm()) < 0.1


@pytest.mark.parametrize("T,H,I,E,k", SIZES)
def test_block_is_norm_router_and_layer(T, H, I, E, k):
    moe = need_gpu()
    from mixture_experts_routing_token_gb300.fp8_layer import Fp8Experts
    x, _, w13, w2 = make(T, H, I, E)
    residual, router = torch.randn(T, H, device=DEV).bfloat16(), torch.randn(E, H, device=DEV) * H ** -0.5
    norm = (1 + 0.1 * torch.randn(H, device=DEV)).bfloat16()
    layer = Fp8Experts(w13, w2, norm=norm)
    out, h = layer.block(x, residual, lambda n: n.float() @ router.t(), k)
    assert torch.equal(h, (x.float() + residual.float()).bfloat16())
    codes, scales, _, n = moe.moe_rms_norm_fp8(x, norm, residual=residual, want_normed=True)
    weights, indices = moe.moe_gating_softmax_topk(n.float() @ router.t(), k)
    r = moe.moe_align_by_expert(indices, weights, E)
    rows = moe.moe_fp8_gather_rows(codes, scales, r["sorted_token_ids"], r["offsets"])
    act = moe.moe_fp8_grouped_gemm(*rows, *layer.w13, r["offsets"], activation="silu_and_mul")
    y = moe.moe_fp8_grouped_gemm(*moe.moe_fp8_quantize(act), *layer.w2, r["offsets"])
    assert torch.equal(out, moe.moe_ep_combine(y, weights, r["reverse_indices"], r["offsets"]))
    # in place, on another stream
    keep = residual.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out2, h2 = layer.block(x, keep, lambda n: n.float() @ router.t(), k, residual_out=keep, stream=s)
    torch.cuda.synchronize()
    assert h2 is keep and torch.equal(h2, h) and torch.equal(out2, out)


def test_layer_in_a_graph_on_a_stream():
    need_gpu()
    from mixture_experts_routing_token_gb300.fp8_layer import Fp8Experts
    x, _, w13, w2 = make(40, 128, 128, 8)
    router = torch.randn(8, 128, device=DEV)
    layer = Fp8Experts(w13, w2, norm=torch.ones(128, device=DEV, dtype=torch.bfloat16))
    call = lambda x, r, out: layer.block(x, r, lambda n: n.float() @ router.t(), 2, residual_out=r, out=out)  # noqa: E731
    r0 = torch.randn(40, 128, device=DEV).bfloat16()
    want = torch.empty_like(x)
    r1 = r0.clone()
    call(x, r1, want)
    x2, r2, out = torch.zeros_like(x), torch.zeros_like(x), torch.empty_like(x)
    call(x2, r2, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(x2, r2, out)
    x2.copy_(x)
    r2.copy_(r0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(r2, r1)


@pytest.mark.parametrize("handle", [False, True])
def test_memory_of_calls_on_another_stream(handle):
    """Neither stream meets the other's blocks: what the current stream has given back is still read there, and what the
    call drops is given out again while it runs."""
    need_gpu()
    from mixture_experts_routing_token_gb300.fp8_layer import Fp8Experts
    T, H, M, E, K = 300, 128, 96, 8, 2
    hidden, logits, w13, w2 = make(T, H, M, E)
    layer = Fp8Experts(w13, w2)
    want = layer(hidden, logits, K)
    s = torch.cuda.Stream()
    sizes = [4 * E, 4 * (E + 1), 4 * T * K, T * H, 4 * T, T * K * H, T * K * M, T * K * M * 2, T * K * H * 2, 1 << 16]
    torch.cuda.synchronize()
    mine = [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(3)]
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(4000000)
    copies = [m.clone() for m in mine]
    del mine
    got = layer(hidden, logits, K, stream=s.cuda_stream if handle else s)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all((c == 7).all() for c in copies)


def test_layer_without_tokens():
    need_gpu()
    from mixture_experts_routing_token_gb300.fp8_layer import Fp8Experts
    hidden, logits, w13, w2 = make(1, 64, 64, 4)
    assert Fp8Experts(w13, w2)(hidden[:0], logits[:0], 2).shape == (0, 64)


def test_layer_refusals():
    need_gpu()
    from mixture_experts_routing_token_gb300.fp8_layer import Fp8Experts
    hidden, logits, w13, w2 = make(3, 64, 64, 4)
    with pytest.raises(ValueError, match="w13 must be"):
        Fp8Experts(w13, w2[:, :, :32].contiguous())
    with pytest.raises(ValueError, match="multiples of 16"):
        Fp8Experts(w13[:, :80].contiguous(), w2[:, :, :40].contiguous())
    with pytest.raises(ValueError, match="norm must be"):
        Fp8Experts(w13, w2, norm=torch.ones(64, device=DEV))
    layer = Fp8Experts(w13, w2)
    with pytest.raises(ValueError, match="router_logits"):
        layer(hidden, logits[:, :2].contiguous(), 2)
    with pytest.raises(ValueError, match="norm's weight"):
        layer.block(hidden, hidden, lambda n: logits, 2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_training_step(dtype):
    """out = combine(gather(hidden) w^T) and all its gradients by the calls, against the oracles; every rounding is half a
    step of the type: y, then the sum; d_y, then d_x or d_w, then the sum over k."""
    moe = need_gpu()
    T, k, E, H, N = 150, 3, 6, 72, 40
    g = torch.Generator().manual_seed(3)
    hidden, w, d_out = (torch.randn(*s, generator=g).to(dtype) for s in ((T, H), (E, N, H), (T, N)))
    logits = torch.randn(T, E, generator=g).to(DEV)
    weights, indices = moe.moe_gating_softmax_topk(logits, k)
    indices[::7, 1] = -1                                    # slots that no expert takes
    r = moe.moe_align_by_expert(indices, weights, E)
    rev, off = r["reverse_indices"], r["offsets"]
    hg, wg, dg = hidden.to(DEV), w.to(DEV), d_out.to(DEV)
    x = moe.moe_gather_rows(hg, r["sorted_token_ids"], off, k)
    y = moe.moe_grouped_gemm(x, wg, off)
    out = moe.moe_ep_combine(y, weights, rev, off)
    d_y, d_weights = moe.moe_ep_combine_backward(dg, y, weights, rev, off)
    d_x, d_w = moe.moe_grouped_gemm_backward(x, wg, off, d_y)
    d_hidden = moe.moe_gather_rows_backward(d_x, rev, off, k)
    n, reverse, offs = int(off[-1]), rev.cpu().numpy(), off.cpu().numpy()
    h64, w64, d64, p64 = hidden.double().numpy(), w.double().numpy(), d_out.double().numpy(), weights.double().cpu().numpy()
    ox = sorted_rows.gather(h64, reverse, n, k)
    oy = grouped.grouped_gemm(ox, w64, offs)
    o_dy, o_dw = sorted_rows.combine_backward(d64, oy, p64, reverse, n)
    o_dx, o_w = grouped.grouped_gemm_backward(ox, w64, offs, o_dy)
    pairs = [(out, sorted_rows.combine(oy, p64, reverse, n)), (d_weights, o_dw), (d_w, o_w),
             (d_hidden, sorted_rows.gather_backward(o_dx, reverse, n, T, k))]
    for got, want in pairs:
        # three roundings in a row and float32 sums of up to 150 terms (2^-16 for both together in float32)
        tol = 3 * torch.finfo(dtype).eps / 2 + 2.0 ** -16
        diff = got.double().cpu().numpy() - want
        assert np.linalg.norm(diff) <= tol * np.linalg.norm(want)
