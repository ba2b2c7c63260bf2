"""A call whose tensors lie on another device than the current one is refused before the library hears of it (the
library launches on the current device). Checked without a GPU."""
import pytest

import mixture_experts_routing_token_gb300._binding as binding
from host_stand_ins import CALLS, Lib, OnGpu, forget_sizes


class Stream:
    cuda_stream = 4096


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_device_are_refused(monkeypatch, name):
    import torch
    empty, lib = torch.empty, Lib()
    monkeypatch.setattr(binding, "_new", lambda shape, dtype, index, stream: empty(shape, dtype=dtype).as_subclass(OnGpu))
    monkeypatch.setattr(binding, "lib", lambda: lib)
    forget_sizes()
    monkeypatch.setattr(binding, "_current_device", lambda: 0, raising=False)
    CALLS[name](Stream())
    assert len(lib.called) == 1
    monkeypatch.setattr(binding, "_current_device", lambda: 1, raising=False)
    with pytest.raises(ValueError, match="cuda:0.*current device is cuda:1"):
        CALLS[name](Stream())
    assert len(lib.called) == 1
    forget_sizes()
