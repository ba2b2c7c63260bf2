"""Sizes that the library's 32-bit arguments cannot hold are refused by the grouped and 4-bit calls. Checked without a
GPU."""
import pytest
import torch

import mixture_experts_routing_token_gb300._binding as binding
from host_stand_ins import B, I, U, Lib, OnGpu, forget_sizes, gpu

MANY = 2 ** 32 + 2      # 2 in 32 bits


def meta(*shape, dtype=B):
    """A tensor of any size without memory."""
    return gpu(*shape, dtype=dtype, device="meta")


WIDE = {
    "product": lambda: binding.moe_grouped_gemm(meta(MANY, 1), meta(2, 1, 1), gpu(3, dtype=I)),
    "product_columns": lambda: binding.moe_grouped_gemm(meta(2, 1), meta(2, MANY, 1), gpu(3, dtype=I)),
    "gradients": lambda: binding.moe_grouped_gemm_backward(meta(MANY, 1), meta(2, 1, 1), gpu(3, dtype=I), meta(MANY, 1)),
    "quantize": lambda: binding.moe_mxfp4_quantize(meta(MANY, 32)),
    "quantize_rows": lambda: binding.moe_mxfp4_quantize(meta(4, 32), rows=meta(MANY, dtype=I)),
    "dequantize": lambda: binding.moe_mxfp4_dequantize(meta(MANY, 16, dtype=U), meta(MANY, 1, dtype=U)),
    "product4": lambda: binding.moe_mxfp4_grouped_gemm(meta(MANY, 16, dtype=U), meta(MANY, 1, dtype=U), meta(2, 8, 16, dtype=U),
                                                       meta(2, 8, 1, dtype=U), gpu(3, dtype=I)),
}


@pytest.mark.parametrize("name", WIDE)
def test_sizes_past_32_bits_are_refused(monkeypatch, name):
    lib = Lib()
    empty = torch.empty
    monkeypatch.setattr(binding, "_new", lambda shape, dtype, index, stream: empty(shape, dtype=dtype, device="meta").as_subclass(OnGpu))
    monkeypatch.setattr(binding, "lib", lambda: lib)
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    monkeypatch.setattr(binding, "_raw", lambda stream, index: 0)
    forget_sizes()
    with pytest.raises(ValueError, match="below 2\\^31"):
        WIDE[name]()
    assert not lib.called
    forget_sizes()


def test_workspace_sizes_refuse_what_does_not_fit():
    for call in (lambda: binding.moe_grouped_gemm_workspace_size(1, MANY, 1, 1, 1),
                 lambda: binding.moe_grouped_gemm_backward_workspace_size(1, 1, 1, MANY, 1),
                 lambda: binding.moe_mxfp4_quantize_workspace_size(1, 32, True, MANY),
                 lambda: binding.moe_mxfp4_grouped_gemm_workspace_size(MANY, 32, 1, 1)):
        with pytest.raises(ValueError, match="below 2\\^31"):
            call()
