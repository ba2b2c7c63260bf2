"""What the grouped products and the 4-bit calls refuse, at the C boundary and in the binding (no GPU)."""
import ctypes

import pytest
import torch

BAD, WORKSPACE = 1, 4


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routing_token_gb300 as moe
    from mixture_experts_routing_token_gb300.build import build
    build()
    moe.lib()
    return moe


def err(moe):
    return moe.lib().moe_last_error().decode()


def test_grouped_gemm_sizes_and_types(moe):
    f = moe.lib().moe_grouped_gemm
    one = ctypes.c_void_p(16)          # never read: every call is refused on the host
    call = lambda x=one, dtype=1, S=4, K=8, N=8, E=2, off=one, y=one: f(x, one, dtype, S, K, N, E, off, y, None, 0, None, None)  # noqa: E731
    assert call(dtype=3) == BAD and "dtype" in err(moe)
    assert call(S=-1) == BAD and call(K=-1) == BAD and call(N=-1) == BAD
    assert call(E=0) == BAD and call(E=1025) == BAD and "E must be" in err(moe)
    assert call(E=1024, N=1 << 22) == BAD and "too large" in err(moe)
    assert call(x=None) == BAD and "x is null" in err(moe)
    assert call(x=ctypes.c_void_p(8)) == BAD and "aligned" in err(moe)
    assert call(x=None, S=0, K=0, N=0, off=None) == BAD and "offsets" in err(moe)


def test_backward_sizes_and_types(moe):
    f = moe.lib().moe_grouped_gemm_backward
    assert f(None, None, None, 7, 1, 1, 1, 1, None, None, None, None, 0, None, None) == BAD
    assert f(None, None, None, 1, 1, 1, -1, 1, None, None, None, None, 0, None, None) == BAD
    assert f(None, None, None, 1, 1, 8, 8, 1, None, None, None, None, 0, None, None) == BAD and "d_y is null" in err(moe)


def test_workspace_sizes(moe):
    for f in (moe.moe_grouped_gemm_workspace_size, moe.moe_grouped_gemm_backward_workspace_size):
        assert f(moe.MOE_BF16, 100, 64, 128, 4) == 0 and f(moe.MOE_F16, 100, 63, 128, 4) >= (100 + 4 * 128) * 64 * 2
        assert f(moe.MOE_F32, 100, 63, 127, 4) == 0 and f(moe.MOE_F32, 2000, 517, 1030, 8) >= 6 * (2000 + 8 * 1030) * 517
        assert f(moe.MOE_BF16, -1, 64, 64, 4) == 0


@pytest.mark.parametrize("empty", ["S", "K", "N", "SK", "KN", "SN", "SKN"])
def test_empty_calls_need_no_workspace(moe, empty):
    S, K, N = (0 if c in empty else n for c, n in zip("SKN", (50, 640, 96)))
    assert moe.moe_grouped_gemm_workspace_size(moe.MOE_F32, S, K, N, 3) == 0
    assert moe.moe_grouped_gemm_backward_workspace_size(moe.MOE_F32, S, K, N, 3) == 0
    for dtype in (moe.MOE_BF16, moe.MOE_F16):       # rows of 640 or 96 values need no padded copies
        assert moe.moe_grouped_gemm_workspace_size(dtype, S, K, N, 3) == 0
        assert moe.moe_grouped_gemm_backward_workspace_size(dtype, S, K, N, 3) == 0
    moe.moe_mxfp4_grouped_gemm_workspace_size(S, K, N, 3)
    moe.moe_mxfp4_quantize_workspace_size(S, K, 1, S)


def test_largest_sizes_are_answered(moe):
    big = 2 ** 31 - 1
    for dtype in (moe.MOE_F32, moe.MOE_BF16):
        for S, K, N in ((big, 64, 64), (64, big, 64), (64, 64, big)):
            moe.moe_grouped_gemm_workspace_size(dtype, S, K, N, 3)
            moe.moe_grouped_gemm_backward_workspace_size(dtype, S, K, N, 3)


def test_quantize_sizes_and_types(moe):
    f = moe.lib().moe_mxfp4_quantize
    one = ctypes.c_void_p(16)
    assert f(one, 5, 4, 32, None, 4, one, one, None, 0, None, None) == BAD
    assert f(one, 0, 4, 33, None, 4, one, one, None, 0, None, None) == BAD and "multiple of 32" in err(moe)
    assert f(one, 0, 4, 32, None, 5, one, one, None, 0, None, None) == BAD and "R must equal T" in err(moe)
    assert f(one, 0, -4, 32, one, 5, one, one, None, 0, None, None) == BAD
    assert f(None, 0, 0, 32, None, 0, None, None, None, 0, None, None) == 0
    g = moe.lib().moe_mxfp4_dequantize
    assert g(one, one, 4, 48, 1, one, None) == BAD and g(one, one, -1, 32, 1, one, None) == BAD
    assert g(None, None, 0, 32, 2, None, None) == 0


def test_mxfp4_product_sizes_and_types(moe):
    f = moe.lib().moe_mxfp4_grouped_gemm
    one = ctypes.c_void_p(16)
    call = lambda K=64, N=8, act=0, dt=1: f(one, one, one, one, 4, K, N, 2, None, act, dt, one, None, 0, None, None)  # noqa: E731
    assert call(K=40) == BAD and "multiple of 32" in err(moe)
    assert call(act=2) == BAD and "activation" in err(moe)
    assert call(act=1, N=7) == BAD and "even" in err(moe)
    assert call(dt=9) == BAD


def test_binding_wants_device_tensors(moe):
    x, w, off = torch.zeros(4, 32), torch.zeros(2, 8, 32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_grouped_gemm(x, w, off)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_grouped_gemm_backward(x, w, off, torch.zeros(4, 8))
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_mxfp4_quantize(x)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_mxfp4_dequantize(x.byte(), x.byte())
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_mxfp4_grouped_gemm(x.byte(), x.byte(), w.byte(), w.byte(), off)
