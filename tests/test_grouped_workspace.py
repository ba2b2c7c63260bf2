"""Workspace sizes of the 4-bit product go by the activation, named as in the call or by the library's code (no GPU)."""
import ctypes

import pytest


@pytest.mark.parametrize("N", [225, 224, 450, 1000])
def test_size_by_activation(N):
    import mixture_experts_routing_token_gb300 as moe
    from mixture_experts_routing_token_gb300.build import build
    build()
    size = moe.moe_mxfp4_grouped_gemm_workspace_size
    f = moe.lib().moe_mxfp4_grouped_gemm_workspace_size
    for named, code in ((None, moe.MOE_ACT_NONE), ("silu_and_mul", moe.MOE_ACT_SILU_AND_MUL)):
        assert size(1000, 64, N, 3, named) == size(1000, 64, N, 3, code) == f(1000, 64, N, 3, code)
    with pytest.raises(ctypes.ArgumentError):
        size(1000, 64, N, 3, "gelu")
