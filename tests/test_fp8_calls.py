"""The 8-bit calls and the sorted rows' gradients without a GPU: where their memory comes from, what the binding and the C
boundary refuse."""
import ctypes

import pytest
import torch

import mixture_experts_routing_token_gb300._binding as binding
from host_stand_ins import B, E, F, H, I, K, M, T, Lib, OnGpu, forget_sizes, gpu

BAD, WORKSPACE = 1, 4
F8 = torch.float8_e4m3fn
MANY = 2 ** 32 + 16


def eight(*shape, block_rows=1, device=None):
    lead = shape[:-1] if block_rows == 1 else (*shape[:-2], -(-shape[-2] // 128))
    return gpu(*shape, dtype=F8, device=device), gpu(*lead, -(-shape[-1] // 128), device=device)


CALLS = {
    "quantize": lambda s: binding.moe_fp8_quantize(gpu(T, H), stream=s),
    "quantize_blocks": lambda s: binding.moe_fp8_quantize(gpu(E, 2 * M, H, dtype=B), block_rows=128, stream=s),
    "dequantize": lambda s: binding.moe_fp8_dequantize(*eight(T, H), stream=s),
    "norm": lambda s: binding.moe_rms_norm_fp8(gpu(T, H), gpu(H), residual=gpu(T, H), want_normed=True, stream=s),
    "gather": lambda s: binding.moe_fp8_gather_rows(*eight(T, H), gpu(T * K, dtype=I), gpu(E + 1, dtype=I), stream=s),
    "product": lambda s: binding.moe_fp8_grouped_gemm(*eight(T, H), *eight(E, M, H, block_rows=128), gpu(E + 1, dtype=I), stream=s),
    "gather_gradient": lambda s: binding.moe_gather_rows_backward(gpu(T * K, H), gpu(T * K, dtype=I), gpu(E + 1, dtype=I), K, stream=s),
    "combine_gradient": lambda s: binding.moe_ep_combine_backward(gpu(T, H), gpu(T * K, H), gpu(T, K), gpu(T * K, dtype=I),
                                                                  gpu(E + 1, dtype=I), stream=s),
}


class Stream:
    cuda_stream = 4096


@pytest.fixture
def calls(monkeypatch):
    """(stream, bytes) of the allocations since, and the library's stand-in."""
    made, lib, empty = [], Lib(), torch.empty

    def new(shape, dtype, index, stream):
        t = empty(shape, dtype=dtype).as_subclass(OnGpu)
        made.append((stream, t.numel() * t.element_size()))
        return t

    monkeypatch.setattr(binding, "_new", new)
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None, **more:
                        empty(shape, dtype=dtype, device=device, **more) if more else new(shape, dtype, 0, "current"))
    monkeypatch.setattr(binding, "lib", lambda: lib)
    monkeypatch.setattr(binding, "_current_device", lambda: 0, raising=False)
    forget_sizes()
    yield made, lib
    forget_sizes()


@pytest.mark.parametrize("name", CALLS)
def test_memory_comes_from_the_calls_stream(calls, name):
    made, _ = calls
    s = Stream()
    CALLS[name](s)
    assert made and all(stream is s for stream, _ in made)


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_device_are_refused(monkeypatch, calls, name):
    _, lib = calls
    CALLS[name](Stream())
    assert len(lib.called) == 1
    monkeypatch.setattr(binding, "_current_device", lambda: 1, raising=False)
    with pytest.raises(ValueError, match="cuda:0.*current device is cuda:1"):
        CALLS[name](Stream())
    assert len(lib.called) == 1


def test_the_layer_takes_all_its_memory_from_its_stream(calls):
    made, _ = calls
    from mixture_experts_routing_token_gb300.fp8_layer import Fp8Experts
    s = Stream()
    layer = Fp8Experts(gpu(E, 2 * M, H), gpu(E, H, M), stream=s)
    layer(gpu(T, H, dtype=B), gpu(T, E), K, stream=s)
    assert len(made) >= 15 and all(stream is s for stream, _ in made)


def meta(*shape, dtype=F):
    return gpu(*shape, dtype=dtype, device="meta")


WIDE = {
    "quantize": lambda: binding.moe_fp8_quantize(meta(MANY, 16)),
    "quantize_columns": lambda: binding.moe_fp8_quantize(meta(1, MANY)),
    "quantize_blocks": lambda: binding.moe_fp8_quantize(meta(1 << 16, 1 << 15, 16), block_rows=128),
    "dequantize": lambda: binding.moe_fp8_dequantize(*eight(MANY, 16, device="meta")),
    "norm": lambda: binding.moe_rms_norm_fp8(meta(MANY, 16), meta(16)),
    "gather": lambda: binding.moe_fp8_gather_rows(*eight(4, 16, device="meta"), meta(MANY, dtype=I), gpu(3, dtype=I)),
    "product": lambda: binding.moe_fp8_grouped_gemm(*eight(MANY, 16, device="meta"), *eight(2, 16, 16, block_rows=128), gpu(3, dtype=I)),
    "product_columns": lambda: binding.moe_fp8_grouped_gemm(*eight(4, 16), *eight(2, MANY, 16, block_rows=128, device="meta"), gpu(3, dtype=I)),
    "gather_gradient": lambda: binding.moe_gather_rows_backward(meta(MANY, 1), meta(MANY, dtype=I), gpu(3, dtype=I), 2),
    "combine_gradient": lambda: binding.moe_ep_combine_backward(meta(MANY, 1), meta(MANY, 1), meta(MANY, 1), meta(MANY, dtype=I), gpu(3, dtype=I)),
}


@pytest.mark.parametrize("name", WIDE)
def test_sizes_past_32_bits_are_refused(monkeypatch, calls, name):
    _, lib = calls
    monkeypatch.setattr(binding, "_raw", lambda stream, index: 0)
    with pytest.raises(ValueError, match="below 2\\^31"):
        WIDE[name]()
    assert not lib.called


REFUSED = {
    "width": (lambda: binding.moe_fp8_quantize(gpu(T, 24)), "multiple of 16"),
    "block_rows": (lambda: binding.moe_fp8_quantize(gpu(T, H), block_rows=64), "block_rows"),
    "one_dimension": (lambda: binding.moe_fp8_quantize(gpu(H), block_rows=128), "N, K"),
    "integers": (lambda: binding.moe_fp8_quantize(gpu(T, H, dtype=I)), "unsupported dtype"),
    "strided": (lambda: binding.moe_fp8_quantize(gpu(H, T * 16).t()), "contiguous"),
    "codes_shape": (lambda: binding.moe_fp8_quantize(gpu(T, H), codes=gpu(T + 1, H, dtype=F8)), "codes must have shape"),
    "scales_shape": (lambda: binding.moe_fp8_dequantize(gpu(T, H, dtype=F8), gpu(T, 2)), "scales must have shape"),
    "bytes": (lambda: binding.moe_fp8_dequantize(gpu(T, H, dtype=torch.uint8), gpu(T, 1)), "float8_e4m3fn"),
    "norm_weight": (lambda: binding.moe_rms_norm_fp8(gpu(T, H), gpu(H + 16)), "weight"),
    "norm_types": (lambda: binding.moe_rms_norm_fp8(gpu(T, H), gpu(H, dtype=B)), "weight must be torch.float32"),
    "norm_residual": (lambda: binding.moe_rms_norm_fp8(gpu(T, H), gpu(H), residual=gpu(T + 1, H)), "residual as x"),
    "norm_residual_out": (lambda: binding.moe_rms_norm_fp8(gpu(T, H), gpu(H), residual_out=gpu(T, H)), "needs a residual"),
    "gather_scales": (lambda: binding.moe_fp8_gather_rows(gpu(T, H, dtype=F8), gpu(T, 2), gpu(3, dtype=I), gpu(3, dtype=I)), "shapes"),
    "gather_ids": (lambda: binding.moe_fp8_gather_rows(*eight(T, H), gpu(3), gpu(3, dtype=I)), "sorted_token_ids must be torch.int32"),
    "product_width": (lambda: binding.moe_fp8_grouped_gemm(*eight(T, 24), *eight(E, M, 24, block_rows=128), gpu(E + 1, dtype=I)), "multiple of 16"),
    "product_scales": (lambda: binding.moe_fp8_grouped_gemm(*eight(T, H), *eight(E, M, H), gpu(E + 1, dtype=I)), "shapes"),
    "product_gate": (lambda: binding.moe_fp8_grouped_gemm(*eight(T, H), *eight(E, 48, H, block_rows=128), gpu(E + 1, dtype=I),
                                                          activation="silu_and_mul"), "multiple of 32"),
    "product_activation": (lambda: binding.moe_fp8_grouped_gemm(*eight(T, H), *eight(E, M, H, block_rows=128), gpu(E + 1, dtype=I),
                                                                activation="gelu"), "activation"),
    "product_offsets": (lambda: binding.moe_fp8_grouped_gemm(*eight(T, H), *eight(E, M, H, block_rows=128), gpu(E, dtype=I)), "shapes"),
    "gradient_k": (lambda: binding.moe_gather_rows_backward(gpu(T * K, H), gpu(T * K, dtype=I), gpu(E + 1, dtype=I), 5), "shapes"),
    "gradient_reverse": (lambda: binding.moe_gather_rows_backward(gpu(T * K, H), gpu(T, dtype=I), gpu(E + 1, dtype=I), K), "shapes"),
    "gradient_y": (lambda: binding.moe_ep_combine_backward(gpu(T, H), None, gpu(T, K), gpu(T * K, dtype=I), gpu(E + 1, dtype=I)), "y_sorted"),
    "gradient_types": (lambda: binding.moe_ep_combine_backward(gpu(T, H), gpu(T * K, H, dtype=B), gpu(T, K), gpu(T * K, dtype=I),
                                                               gpu(E + 1, dtype=I)), "y_sorted must be torch.float32"),
    "gradient_weights": (lambda: binding.moe_ep_combine_backward(gpu(T, H), gpu(T * K, H), gpu(T, K + 1), gpu(T * K, dtype=I),
                                                                 gpu(E + 1, dtype=I)), "shapes"),
    "host": (lambda: binding.moe_fp8_quantize(torch.zeros(T, H)), "CUDA"),
}


@pytest.mark.parametrize("name", REFUSED)
def test_the_binding_refuses(monkeypatch, calls, name):
    _, lib = calls
    monkeypatch.setattr(binding, "_raw", lambda stream, index: 0)
    call, match = REFUSED[name]
    with pytest.raises(ValueError, match=match):
        call()
    assert not lib.called


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routing_token_gb300 as moe
    from mixture_experts_routing_token_gb300.build import build
    build()
    moe.lib()
    return moe


one = ctypes.c_void_p(16)          # never read: every call is refused on the host


def err(moe):
    return moe.lib().moe_last_error().decode()


def test_c_quantize(moe):
    f, g = moe.lib().moe_fp8_quantize, moe.lib().moe_fp8_dequantize
    assert f(one, 3, 1, 4, 16, 1, one, one, None) == BAD and "dtype" in err(moe)
    assert f(one, 0, 1, 4, 24, 1, one, one, None) == BAD and "multiple of 16" in err(moe)
    assert f(one, 0, 1, 4, 16, 2, one, one, None) == BAD and "block_rows" in err(moe)
    assert f(one, 0, -1, 4, 16, 1, one, one, None) == BAD and f(one, 0, 1, 4, -16, 1, one, one, None) == BAD
    assert f(one, 0, 1 << 16, 1 << 16, 16, 1, one, one, None) == BAD and "2^31" in err(moe)
    assert f(one, 0, 1 << 24, 64, 1 << 15, 128, one, one, None) == BAD and "too large" in err(moe)
    assert f(None, 0, 1, 4, 16, 1, one, one, None) == BAD and "x is null" in err(moe)
    assert f(ctypes.c_void_p(8), 0, 1, 4, 16, 1, one, one, None) == BAD and "aligned" in err(moe)
    assert f(None, 0, 0, 4, 16, 1, None, None, None) == 0 and f(None, 0, 1, 4, 0, 1, None, None, None) == 0
    assert g(one, one, 1, 4, 24, 1, 0, one, None) == BAD and g(one, one, 1, 4, 16, 1, 5, one, None) == BAD
    assert g(None, None, 0, 4, 16, 128, 0, None, None) == 0


def test_c_norm(moe):
    f = moe.lib().moe_rms_norm_fp8
    call = lambda x=one, r=None, dt=0, T=4, H=64, eps=1e-6, ro=None: f(x, r, one, dt, T, H, eps, one, one, ro, None, None)  # noqa: E731
    assert call(dt=4) == BAD and call(T=-1) == BAD and call(H=40) == BAD and "multiple of 16" in err(moe)
    assert call(eps=-1.0) == BAD and "eps" in err(moe) and call(eps=float("nan")) == BAD
    assert call(r=one) == BAD and "together" in err(moe) and call(ro=one) == BAD
    assert call(x=None) == BAD and "x is null" in err(moe)
    assert f(None, None, None, 0, 0, 64, 0.0, None, None, None, None, None) == 0


def test_c_gather_and_product(moe):
    g = moe.lib().moe_fp8_gather_rows
    call = lambda T=4, H=64, E=2, S=8, c=one: g(c, one, one, one, T, H, E, S, one, one, None, None)  # noqa: E731
    assert call(T=-1) == BAD and call(S=-1) == BAD and call(E=0) == BAD and call(E=1025) == BAD and call(H=8) == BAD
    assert call(c=None) == BAD and "codes is null" in err(moe)
    f = moe.lib().moe_fp8_grouped_gemm
    call = lambda S=4, K=64, N=32, E=2, act=0, dt=1, x=one: f(x, one, one, one, S, K, N, E, one, act, dt, one, None, None)  # noqa: E731
    assert call(K=40) == BAD and "multiple of 16" in err(moe)
    assert call(act=2) == BAD and "activation" in err(moe)
    assert call(act=1, N=48) == BAD and "multiple of 16" in err(moe)
    assert call(dt=9) == BAD and call(E=0) == BAD and call(S=-1) == BAD and call(E=1024, N=1 << 22) == BAD
    assert call(x=None) == BAD and "x_codes is null" in err(moe)


def test_c_gradients(moe):
    L = moe.lib()
    f = L.moe_gather_rows_backward
    call = lambda dt=1, T=4, H=8, E=4, k=2, x=one, ws=None, nb=0: f(x, one, one, dt, T, H, E, k, one, ws, nb, None, None)  # noqa: E731
    assert call(dt=7) == BAD and call(H=0) == BAD and call(k=5) == BAD and call(T=-1) == BAD and call(k=33, E=64) == BAD
    assert call(x=None) == BAD and "d_x_sorted is null" in err(moe)
    assert call(H=2 ** 31 - 64) == BAD and "H must be" in err(moe)
    assert f(None, None, one, 1, 0, 8, 4, 2, None, None, 0, None, None) == BAD      # offsets: not device memory
    g = L.moe_ep_combine_backward
    call = lambda dt=1, T=4, H=8, E=4, k=2, d=one: g(d, one, one, one, one, dt, T, k, H, E, one, one, None, 0, None, None)  # noqa: E731
    assert call(dt=7) == BAD and call(H=0) == BAD and call(k=5) == BAD and call(T=-1) == BAD
    assert call(d=None) == BAD and "d_out is null" in err(moe)
    assert call(H=2 ** 31 - 1) == BAD and "H must be" in err(moe)


def test_workspace_sizes(moe):
    for f in (moe.moe_gather_rows_backward_workspace_size, moe.moe_ep_combine_backward_workspace_size):
        assert f(0, 2) == 0 and f(8, 2) == 0 and f(100000, 8) >= 4 * 800000 and f(-1, 2) == 0
        with pytest.raises(ValueError, match="below 2\\^31"):
            f(MANY, 1)
