"""Where the memory of a call on a caller's stream comes from, checked without a GPU: tensors in host memory that say
they lie on one, and a library that answers every call with 0."""
import pytest
import torch

import mixture_experts_routing_token_gb300._binding as binding


class OnGpu(torch.Tensor):
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 0))

    def get_device(self):
        return 0


class Stream:
    cuda_stream = 4096


class Lib:
    def __getattr__(self, name):
        return lambda *args: 512 if name.endswith("_size") else 0


def gpu(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


@pytest.fixture
def calls(monkeypatch):
    """Allocations of the calls made since, as (stream, bytes); one that names no stream has the stream "current"."""
    made = []
    empty = torch.empty

    def new(shape, dtype, index, stream):
        t = empty(shape, dtype=dtype).as_subclass(OnGpu)
        made.append((stream, t.numel() * t.element_size()))
        return t

    def direct(shape, dtype=None, device=None):
        return new(shape, dtype, 0, "current")

    monkeypatch.setattr(binding, "_new", new)
    monkeypatch.setattr(torch, "empty", direct)
    monkeypatch.setattr(binding, "lib", lambda: Lib())
    sizes = [f for f in vars(binding).values() if hasattr(f, "cache_clear") and f.__name__.endswith("_size")]
    for f in sizes:
        f.cache_clear()
    yield made
    for f in sizes:
        f.cache_clear()


I, F, B = torch.int32, torch.float32, torch.bfloat16
T, K, E, H, M = 6, 2, 4, 64, 32      # tokens, experts a token, experts, hidden and intermediate width


def aligned():
    return (gpu(E, dtype=I), gpu(E + 1, dtype=I), gpu(T * K, dtype=I), gpu(T * K), gpu(T * K, dtype=I))


def ffn():
    return gpu(T, H, dtype=B), gpu(E, 2 * M, H, dtype=B), gpu(E, H, M, dtype=B)


OLDER = {
    "gating": lambda s: binding.moe_gating_softmax_topk(gpu(T, E), K, stream=s),
    "gating_bf16": lambda s: binding.moe_gating_softmax_topk_bf16(gpu(T, E, dtype=B), K, stream=s),
    "group_limited": lambda s: binding.moe_group_limited_topk(gpu(T, E), K, 2, 1, stream=s),
    "to_multihot": lambda s: binding.moe_indices_to_multihot(gpu(T, K, dtype=I), gpu(T, K), E, stream=s),
    "from_multihot": lambda s: binding.moe_multihot_to_indices(gpu(T, E), gpu(T, E, dtype=I), K, stream=s),
    "align": lambda s: binding.moe_align_by_expert(gpu(T, K, dtype=I), gpu(T, K), E, stream=s),
    "align_noalloc": lambda s: binding.moe_align_by_expert_noalloc(gpu(T, K, dtype=I), gpu(T, K), E, stream=s),
    "ffn": lambda s: binding.moe_grouped_ffn(*ffn(), K, *aligned(), stream=s),
    "ffn_backward": lambda s: binding.moe_grouped_ffn_backward(*ffn(), K, *aligned(), gpu(T, H, dtype=B), stream=s),
    "layer": lambda s: binding.moe_layer_forward(ffn()[0], gpu(T, E), *ffn()[1:], K, stream=s),
    "gather": lambda s: binding.moe_gather_rows(gpu(T, H, dtype=B), gpu(T * K, dtype=I), gpu(E + 1, dtype=I), K, stream=s),
    "receive": lambda s: binding.moe_ep_receive_index(gpu(2, E, dtype=I), 9, stream=s),
    "combine": lambda s: binding.moe_ep_combine(gpu(T * K, H, dtype=B), gpu(T, K), gpu(T * K, dtype=I), gpu(E + 1, dtype=I), stream=s),
}


@pytest.mark.parametrize("name", OLDER)
def test_outputs_and_workspaces_come_from_the_calls_stream(calls, name):
    s = Stream()
    OLDER[name](s)
    assert calls and all(stream is s for stream, _ in calls)


def test_the_4_bit_layer_takes_all_its_memory_from_its_stream(calls):
    from mixture_experts_routing_token_gb300.mxfp4_layer import Mxfp4Experts
    s = Stream()
    layer = Mxfp4Experts(gpu(E, 2 * M, H), gpu(E, H, M), stream=s)
    layer(gpu(T, H, dtype=B), gpu(T, E), K, stream=s)
    assert len(calls) >= 15 and all(stream is s for stream, _ in calls)
