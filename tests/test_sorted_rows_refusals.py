"""What the binding refuses of the forward steps around the expert products: tensors of another type or device and ones
with fewer rows than the call reads (no GPU)."""
import pytest
import torch

import mixture_experts_routing_token_gb300._binding as binding
from host_stand_ins import B, E, H, I, K, T, Lib, OnGpu, gpu

S = T * K


@pytest.fixture
def lib(monkeypatch):
    lib, empty = Lib(), torch.empty
    monkeypatch.setattr(binding, "_new", lambda shape, dtype, index, stream: empty(shape, dtype=dtype).as_subclass(OnGpu))
    monkeypatch.setattr(binding, "lib", lambda: lib)
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    monkeypatch.setattr(binding, "_stream", lambda stream, device: None)
    return lib


def gather(ids=None, offsets=None, k=K, hidden=None):
    return binding.moe_gather_rows(gpu(T, H, dtype=B) if hidden is None else hidden, gpu(S, dtype=I) if ids is None else ids,
                                   gpu(E + 1, dtype=I) if offsets is None else offsets, k)


def combine(y=None, weights=None, reverse=None, offsets=None):
    return binding.moe_ep_combine(gpu(S, H, dtype=B) if y is None else y, gpu(T, K) if weights is None else weights,
                                  gpu(S, dtype=I) if reverse is None else reverse, gpu(E + 1, dtype=I) if offsets is None else offsets)


REFUSED = {
    "long_ids": (lambda: gather(ids=gpu(S, dtype=torch.int64)), "sorted_token_ids must be torch.int32"),
    "host_ids": (lambda: gather(ids=torch.zeros(S, dtype=I)), "sorted_token_ids must be a CUDA tensor"),
    "strided_ids": (lambda: gather(ids=gpu(S, 2, dtype=I)[:, 0]), "sorted_token_ids must be contiguous"),
    "few_ids": (lambda: gather(ids=gpu(S - 1, dtype=I)), "T \\* k = 12"),
    "more_slots": (lambda: gather(k=K + 1), "T \\* k = 18"),
    "long_offsets": (lambda: gather(offsets=gpu(E + 1, dtype=torch.int64)), "offsets must be torch.int32"),
    "few_rows": (lambda: combine(y=gpu(S - 1, H, dtype=B)), "T \\* k = 12"),
    "few_slots": (lambda: combine(reverse=gpu(S - 1, dtype=I)), "T \\* k = 12"),
    "half_weights": (lambda: combine(weights=gpu(T, K, dtype=B)), "topk_weights must be torch.float32"),
    "long_slots": (lambda: combine(reverse=gpu(S, dtype=torch.int64)), "reverse_indices must be torch.int32"),
    "host_offsets": (lambda: combine(offsets=torch.zeros(E + 1, dtype=I)), "offsets must be a CUDA tensor"),
    "no_slots": (lambda: combine(reverse=[0] * S), "reverse_indices must be a CUDA tensor"),
    "wide": (lambda: gather(ids=gpu(2 ** 31, dtype=I, device="meta"), hidden=gpu(2 ** 30, 1, device="meta")), "below 2\\^31"),
}


@pytest.mark.parametrize("name", REFUSED)
def test_refused(lib, name):
    call, match = REFUSED[name]
    with pytest.raises(ValueError, match=match):
        call()
    assert not lib.called


def test_tensors_with_more_room_than_the_call_needs(lib):
    """As they come out of buffers for the largest batch."""
    gather(ids=gpu(S + 5, dtype=I))
    gather(ids=gpu(T, K, dtype=I))
    combine(y=gpu(S + 3, H, dtype=B), reverse=gpu(S + 3, dtype=I))
    assert lib.called == ["moe_gather_rows", "moe_gather_rows", "moe_ep_combine"]
