"""Where the memory of a call on a caller's stream comes from, checked without a GPU."""
import pytest
import torch

import mixture_experts_routing_token_gb300._binding as binding
from host_stand_ins import B, CALLS, E, H, K, M, T, Lib, OnGpu, forget_sizes, gpu


class Stream:
    cuda_stream = 4096


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
    monkeypatch.setattr(binding, "_current_device", lambda: 0, raising=False)
    forget_sizes()
    yield made
    forget_sizes()


@pytest.mark.parametrize("name", CALLS)
def test_outputs_and_workspaces_come_from_the_calls_stream(calls, name):
    s = Stream()
    CALLS[name](s)
    assert calls and all(stream is s for stream, _ in calls)


def test_the_4_bit_layer_takes_all_its_memory_from_its_stream(calls):
    from mixture_experts_routing_token_gb300.mxfp4_layer import Mxfp4Experts
    s = Stream()
    layer = Mxfp4Experts(gpu(E, 2 * M, H), gpu(E, H, M), stream=s)
    layer(gpu(T, H, dtype=B), gpu(T, E), K, stream=s)
    assert len(calls) >= 15 and all(stream is s for stream, _ in calls)
