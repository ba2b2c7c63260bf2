"""Calls on a stream of the caller's while the current stream is busy with memory of its own: neither may meet the
other's blocks."""
import pytest
import torch

from gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu

T, H, M, E, K = 300, 128, 96, 8, 2


def layer_of_4_bits(moe, g):
    from mixture_experts_routing_token_gb300.mxfp4_layer import Mxfp4Experts
    layer = Mxfp4Experts(*(torch.randn(s, generator=g).mul(0.1).to(DEV) for s in ((E, 2 * M, H), (E, H, M))))
    hidden, logits = torch.randn(T, H, generator=g).bfloat16().to(DEV), torch.randn(T, E, generator=g).to(DEV)
    return lambda s: layer(hidden, logits, K, stream=s)


def layer_of_bf16(moe, g):
    w13, w2 = (torch.randn(s, generator=g).mul(0.1).bfloat16().to(DEV) for s in ((E, 2 * M, H), (E, H, M)))
    hidden, logits = torch.randn(T, H, generator=g).bfloat16().to(DEV), torch.randn(T, E, generator=g).to(DEV)
    return lambda s: moe.moe_layer_forward(hidden, logits, w13, w2, K, stream=s)


def routing(moe, g):
    logits, y = torch.randn(T, E, generator=g).to(DEV), torch.randn(T * K, H, generator=g).to(DEV)

    def run(s):
        weights, indices = moe.moe_gating_softmax_topk(logits, K, stream=s)
        r = moe.moe_align_by_expert(indices, weights, E, stream=s)
        return moe.moe_ep_combine(y, weights, r["reverse_indices"], r["offsets"], stream=s)

    return run


@pytest.mark.parametrize("make", [layer_of_4_bits, layer_of_bf16, routing])
@pytest.mark.parametrize("handle", [False, True])
def test_memory_of_calls_on_another_stream(make, handle):
    moe = need_gpu()
    call = make(moe, torch.Generator().manual_seed(1))
    want = call(None)
    s = torch.cuda.Stream()
    sizes = [4 * E, 4 * (E + 1), 4 * T * K, 2 * T * H, 4 * T * H, T * K * H // 2, T * K * M * 2, T * K * H * 2, 1 << 16, 1 << 20]
    torch.cuda.synchronize()
    # what the current stream has given back, but not yet read
    mine = [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(3)]
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(4000000)
    copies = [m.clone() for m in mine]
    del mine
    got = call(s.cuda_stream if handle else s)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all((c == 7).all() for c in copies)
    # what the call has dropped, but not yet read
    with torch.cuda.stream(s):
        torch.cuda._sleep(4000000)
    got = call(s.cuda_stream if handle else s)
    junk = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and junk
