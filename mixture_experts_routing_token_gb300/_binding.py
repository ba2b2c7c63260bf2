"""ctypes binding of ``libmoe_gb300.so`` (the C ABI declared in ``include/moe.h``).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels. PyTorch supplies device memory (output and workspace tensors when
the caller gives none) and the current CUDA stream. There is no CPU or
PyTorch fallback: if the library is missing or a call fails, an exception is
raised.
"""
from __future__ import annotations

import ctypes
import functools
import json
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_gb300.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA, MOE_ERR_WORKSPACE = 0, 1, 2, 3, 4
MOE_F32, MOE_BF16, MOE_F16 = 0, 1, 2
MOE_ACT_NONE, MOE_ACT_SILU_AND_MUL = 0, 1
MOE_STATUS_BAD_INDEX, MOE_STATUS_TIMEOUT = 1, 2
MOE_GROUP_TOPK_GREEDY, MOE_GROUP_TOPK_NOAUX_TC = 0, 1
MOE_MAX_TOPK, MOE_MAX_EXPERTS = 32, 1024
MOE_ALIGN_NOALLOC_SCRATCH_INTS = 65536

_p, _i, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t

# name -> (restype, argtypes); mirrors include/moe.h
SIGNATURES = {
    "moe_gating_softmax_topk": (_i, [_p, _i, _i, _i, _i, _p, _p, _p]),
    "moe_gating_softmax_topk_bf16": (_i, [_p, _i, _i, _i, _i, _p, _p, _p]),
    "moe_group_limited_topk": (_i, [_p, _p, _i, _i, _i, _i, _i, _i, _p, _p, _p]),
    "moe_indices_to_multihot": (_i, [_p, _p, _i, _i, _i, _p, _p, _p, _p]),
    "moe_multihot_to_indices": (_i, [_p, _p, _i, _i, _i, _p, _p, _p]),
    "moe_align_workspace_size": (_sz, [_i, _i, _i]),
    "moe_align_by_expert": (_i, [_p, _p, _i, _i, _i, _p, _p, _p, _p, _p, _p, _sz, _p, _p]),
    "moe_align_by_expert_noalloc": (_i, [_p, _p, _i, _i, _i, _p, _p, _p, _p, _p, _p, _p]),
    "moe_grouped_ffn_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i]),
    "moe_grouped_ffn": (_i, [_p, _p, _p, _i, _i, _i, _i, _i, _i, _p, _p, _p, _p, _p, _p, _p, _sz, _p, _p]),
    "moe_grouped_ffn_backward_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i]),
    "moe_grouped_ffn_backward": (_i, [_p, _p, _p, _i, _i, _i, _i, _i, _i, _p, _p, _p, _p, _p, _p, _p, _p, _p,
                                      _p, _p, _sz, _p, _p]),
    "moe_layer_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i]),
    "moe_layer_forward": (_i, [_p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _p, _p, _p, _p, _sz, _p, _p]),
    "moe_grouped_gemm_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "moe_grouped_gemm": (_i, [_p, _p, _i, _i, _i, _i, _i, _p, _p, _p, _sz, _p, _p]),
    "moe_grouped_gemm_backward_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "moe_grouped_gemm_backward": (_i, [_p, _p, _p, _i, _i, _i, _i, _i, _p, _p, _p, _p, _sz, _p, _p]),
    "moe_mxfp4_quantize_workspace_size": (_sz, [_i, _i, _i, _i]),
    "moe_mxfp4_quantize": (_i, [_p, _i, _i, _i, _p, _i, _p, _p, _p, _sz, _p, _p]),
    "moe_mxfp4_dequantize": (_i, [_p, _p, _i, _i, _i, _p, _p]),
    "moe_mxfp4_grouped_gemm_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "moe_mxfp4_grouped_gemm": (_i, [_p, _p, _p, _p, _i, _i, _i, _i, _p, _i, _i, _p, _p, _sz, _p, _p]),
    "moe_gather_rows": (_i, [_p, _p, _p, _i, _i, _i, _i, _i, _p, _p]),
    "moe_ep_receive_workspace_size": (_sz, [_i, _i]),
    "moe_ep_receive_index": (_i, [_p, _i, _i, _i, _p, _p, _p, _p, _sz, _p]),
    "moe_ep_combine_workspace_size": (_sz, [_i, _i]),
    "moe_ep_combine": (_i, [_p, _p, _p, _p, _i, _i, _i, _i, _i, _p, _p, _sz, _p]),
    "moe_gather_rows_backward_workspace_size": (_sz, [_i, _i]),
    "moe_gather_rows_backward": (_i, [_p, _p, _p, _i, _i, _i, _i, _i, _p, _p, _sz, _p, _p]),
    "moe_ep_combine_backward_workspace_size": (_sz, [_i, _i]),
    "moe_ep_combine_backward": (_i, [_p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _p, _p, _p, _sz, _p, _p]),
    "moe_fp8_quantize": (_i, [_p, _i, _i, _i, _i, _i, _p, _p, _p]),
    "moe_fp8_dequantize": (_i, [_p, _p, _i, _i, _i, _i, _i, _p, _p]),
    "moe_rms_norm_fp8": (_i, [_p, _p, _p, _i, _i, _i, ctypes.c_float, _p, _p, _p, _p, _p]),
    "moe_fp8_gather_rows": (_i, [_p, _p, _p, _p, _i, _i, _i, _i, _p, _p, _p, _p]),
    "moe_fp8_grouped_gemm": (_i, [_p, _p, _p, _p, _i, _i, _i, _i, _p, _i, _i, _p, _p, _p]),
    "moe_set_wait_limit_ns": (ctypes.c_uint64, [ctypes.c_uint64]),
    "moe_profiler_enable": (_i, [_i]),
    "moe_profiler_report": (_i, [ctypes.c_char_p, _sz]),
    "moe_last_error": (ctypes.c_char_p, []),
    "moe_version": (ctypes.c_char_p, []),
}


class MoeError(RuntimeError):
    """A library call returned a non-zero status."""

    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} failed with code {code}: {msg}")
        self.code = code


_lib = None


def lib():
    """Load the library (once). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device):
    if stream is None:
        if _raw_stream is not None:      # the current stream's handle without a Stream object
            return ctypes.c_void_p(_raw_stream(device.index if device.index is not None else
                                               torch.cuda.current_device()))
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(fn, rc):
    if rc != MOE_OK:
        raise MoeError(fn, rc, lib().moe_last_error().decode())


# Index of the current device, without the checks of torch.cuda.current_device: tensors that lie on a GPU came before.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on_current(index, name):
    """The library launches on the current device, so tensors of another one are refused: its kernels would run there
    on this one's addresses."""
    if index != _current_device():
        raise ValueError(f"{name} is on cuda:{index}, but the current device is cuda:{_current_device()}: "
                         f"make the call under torch.cuda.device({index})")


def _dev(t, name, dtype=None):
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise ValueError(f"{name} must be a CUDA tensor")
    _on_current(t.get_device(), name)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    return t


def _dtype_code(t):
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    raise ValueError(f"unsupported dtype {t.dtype}")


_device = functools.lru_cache(maxsize=None)(lambda index: torch.device("cuda", index))


def _new(shape, dtype, index, stream):
    """Memory for a call on ``stream``, from that stream's pool: a block that the current stream has given back may
    still be read by what is queued there, and one of the current stream's that is dropped on return may be given out
    again while the call still runs. The current stream is noted with it, where outputs are used next."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=_device(index))
    handle = int(getattr(stream, "cuda_stream", stream))
    if _raw_stream is not None and handle == _raw_stream(index):
        return torch.empty(shape, dtype=dtype, device=_device(index))
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(handle, device=index)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=_device(index))
    t.record_stream(torch.cuda.current_stream(index))
    return t


def _out(t, shape, dtype, device, name, stream):
    if t is None:
        return _new(shape, dtype, device.index, stream)
    _dev(t, name, dtype)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    return t


def version() -> str:
    return lib().moe_version().decode()


def moe_gating_softmax_topk(logits, k, norm_topk_prob=True, weights=None, indices=None, stream=None):
    """Top-k experts per row of ``logits [T,E]`` (float32) -> (weights [T,k] f32, indices [T,k] i32)."""
    _dev(logits, "logits", torch.float32)
    T, E = logits.shape
    weights = _out(weights, (T, k), torch.float32, logits.device, "weights", stream)
    indices = _out(indices, (T, k), torch.int32, logits.device, "indices", stream)
    _check("moe_gating_softmax_topk", lib().moe_gating_softmax_topk(
        _ptr(logits), T, E, k, int(bool(norm_topk_prob)), _ptr(weights), _ptr(indices),
        _stream(stream, logits.device)))
    return weights, indices


def moe_gating_softmax_topk_bf16(logits, k, norm_topk_prob=True, weights=None, indices=None, stream=None):
    """Top-k experts per row of bf16 ``logits [T,E]`` -> (weights [T,k] f32, indices [T,k] i32)."""
    _dev(logits, "logits", torch.bfloat16)
    T, E = logits.shape
    weights = _out(weights, (T, k), torch.float32, logits.device, "weights", stream)
    indices = _out(indices, (T, k), torch.int32, logits.device, "indices", stream)
    _check("moe_gating_softmax_topk_bf16", lib().moe_gating_softmax_topk_bf16(
        _ptr(logits), T, E, k, int(bool(norm_topk_prob)), _ptr(weights), _ptr(indices),
        _stream(stream, logits.device)))
    return weights, indices


def moe_group_limited_topk(scores, k, n_group, topk_group, method="group_limited_greedy", bias=None,
                           weights=None, indices=None, stream=None):
    """Group-limited top-k of ``scores [T,E]`` f32 -> (weights [T,k] f32, indices [T,k] i32).

    ``method`` is "group_limited_greedy" or "noaux_tc" (needs ``bias [E]`` f32)."""
    _dev(scores, "scores", torch.float32)
    T, E = scores.shape
    code = {"group_limited_greedy": MOE_GROUP_TOPK_GREEDY, "noaux_tc": MOE_GROUP_TOPK_NOAUX_TC}[method]
    if bias is not None:
        _dev(bias, "bias", torch.float32)
    weights = _out(weights, (T, k), torch.float32, scores.device, "weights", stream)
    indices = _out(indices, (T, k), torch.int32, scores.device, "indices", stream)
    _check("moe_group_limited_topk", lib().moe_group_limited_topk(
        _ptr(scores), _ptr(bias), T, E, k, n_group, topk_group, code, _ptr(weights), _ptr(indices),
        _stream(stream, scores.device)))
    return weights, indices


def moe_indices_to_multihot(indices, probs, num_experts, multihot=None, probs_in_multihot=None,
                            position_map=None, stream=None):
    """-> (multihot [T,E] uint8, probs_in_multihot [T,E] f32, position_map [T,E] i32)."""
    _dev(indices, "indices", torch.int32)
    _dev(probs, "probs", torch.float32)
    T, k = indices.shape
    E = int(num_experts)
    d = indices.device
    multihot = _out(multihot, (T, E), torch.uint8, d, "multihot", stream)
    probs_in_multihot = _out(probs_in_multihot, (T, E), torch.float32, d, "probs_in_multihot", stream)
    position_map = _out(position_map, (T, E), torch.int32, d, "position_map", stream)
    _check("moe_indices_to_multihot", lib().moe_indices_to_multihot(
        _ptr(indices), _ptr(probs), T, k, E, _ptr(multihot), _ptr(probs_in_multihot),
        _ptr(position_map), _stream(stream, d)))
    return multihot, probs_in_multihot, position_map


def moe_multihot_to_indices(probs_in_multihot, position_map, k, probs=None, indices=None,
                            with_indices=True, stream=None):
    """-> (probs [T,k] f32, indices [T,k] i32 or None)."""
    _dev(probs_in_multihot, "probs_in_multihot", torch.float32)
    _dev(position_map, "position_map", torch.int32)
    T, E = probs_in_multihot.shape
    d = probs_in_multihot.device
    probs = _out(probs, (T, k), torch.float32, d, "probs", stream)
    if with_indices or indices is not None:
        indices = _out(indices, (T, k), torch.int32, d, "indices", stream)
    _check("moe_multihot_to_indices", lib().moe_multihot_to_indices(
        _ptr(probs_in_multihot), _ptr(position_map), T, E, k, _ptr(probs), _ptr(indices),
        _stream(stream, d)))
    return probs, indices


def moe_align_workspace_size(T, k, E) -> int:
    return int(lib().moe_align_workspace_size(T, k, E))


def moe_align_by_expert(indices, weights, num_experts, out=None, workspace=None, status=None,
                        stream=None):
    """-> dict(counts [E], offsets [E+1], sorted_token_ids, sorted_weights, reverse_indices [T*k])."""
    _dev(indices, "indices", torch.int32)
    _dev(weights, "weights", torch.float32)
    T, k = indices.shape
    E = int(num_experts)
    S = T * k
    d = indices.device
    out = dict(out or {})
    counts = _out(out.get("counts"), (E,), torch.int32, d, "counts", stream)
    offsets = _out(out.get("offsets"), (E + 1,), torch.int32, d, "offsets", stream)
    ids = _out(out.get("sorted_token_ids"), (S,), torch.int32, d, "sorted_token_ids", stream)
    sw = _out(out.get("sorted_weights"), (S,), torch.float32, d, "sorted_weights", stream)
    rev = _out(out.get("reverse_indices"), (S,), torch.int32, d, "reverse_indices", stream)
    need = moe_align_workspace_size(T, k, E)
    if workspace is None and need:
        workspace = _new(need, torch.uint8, d.index, stream)
    _check("moe_align_by_expert", lib().moe_align_by_expert(
        _ptr(indices), _ptr(weights), T, k, E, _ptr(counts), _ptr(offsets), _ptr(ids), _ptr(sw),
        _ptr(rev), _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
        _ptr(status), _stream(stream, d)))
    return dict(counts=counts, offsets=offsets, sorted_token_ids=ids, sorted_weights=sw,
                reverse_indices=rev)


def moe_align_by_expert_noalloc(indices, weights, num_experts, out=None, status=None, stream=None):
    """Align by expert for callers that cannot allocate device memory at call time.

    Same results as :func:`moe_align_by_expert`; the library keeps the scratch in
    a fixed device array of its own (limit: ceil(T*k / 4096) * E <=
    MOE_ALIGN_NOALLOC_SCRATCH_INTS), so no workspace is passed. Calls that
    overlap on the GPU share that array and race. Output tensors are created
    here only when ``out`` does not supply them.
    """
    _dev(indices, "indices", torch.int32)
    _dev(weights, "weights", torch.float32)
    T, k = indices.shape
    E = int(num_experts)
    S = T * k
    d = indices.device
    out = dict(out or {})
    counts = _out(out.get("counts"), (E,), torch.int32, d, "counts", stream)
    offsets = _out(out.get("offsets"), (E + 1,), torch.int32, d, "offsets", stream)
    ids = _out(out.get("sorted_token_ids"), (S,), torch.int32, d, "sorted_token_ids", stream)
    sw = _out(out.get("sorted_weights"), (S,), torch.float32, d, "sorted_weights", stream)
    rev = _out(out.get("reverse_indices"), (S,), torch.int32, d, "reverse_indices", stream)
    _check("moe_align_by_expert_noalloc", lib().moe_align_by_expert_noalloc(
        _ptr(indices), _ptr(weights), T, k, E, _ptr(counts), _ptr(offsets), _ptr(ids), _ptr(sw),
        _ptr(rev), _ptr(status), _stream(stream, d)))
    return dict(counts=counts, offsets=offsets, sorted_token_ids=ids, sorted_weights=sw,
                reverse_indices=rev)


def moe_grouped_ffn_workspace_size(dtype_code, T, H, I, E, k) -> int:
    return int(lib().moe_grouped_ffn_workspace_size(dtype_code, T, H, I, E, k))


def moe_grouped_ffn(hidden, w13, w2, k, counts, offsets, sorted_token_ids, sorted_weights,
                    reverse_indices, out=None, workspace=None, status=None, stream=None):
    """Expert FFN + weighted combine -> out [T,H] (hidden's dtype)."""
    _dev(hidden, "hidden")
    dt = _dtype_code(hidden)
    T, H = hidden.shape
    E, I2, H2 = w13.shape
    I = I2 // 2
    _dev(w13, "w13", hidden.dtype)
    _dev(w2, "w2", hidden.dtype)
    if H2 != H or tuple(w2.shape) != (E, H, I):
        raise ValueError("w13 must be [E, 2I, H] and w2 [E, H, I]")
    d = hidden.device
    out = _out(out, (T, H), hidden.dtype, d, "out", stream)
    need = moe_grouped_ffn_workspace_size(dt, T, H, I, E, k)
    if workspace is None:
        workspace = _new(max(need, 1), torch.uint8, d.index, stream)
    _check("moe_grouped_ffn", lib().moe_grouped_ffn(
        _ptr(hidden), _ptr(w13), _ptr(w2), dt, T, H, I, E, k, _ptr(counts), _ptr(offsets),
        _ptr(sorted_token_ids), _ptr(sorted_weights), _ptr(reverse_indices), _ptr(out),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
        _stream(stream, d)))
    return out


def moe_grouped_ffn_backward_workspace_size(dtype_code, T, H, I, E, k) -> int:
    return int(lib().moe_grouped_ffn_backward_workspace_size(dtype_code, T, H, I, E, k))


def moe_grouped_ffn_backward(hidden, w13, w2, k, counts, offsets, sorted_token_ids, sorted_weights,
                             reverse_indices, d_out, d_hidden=None, d_w13=None, d_w2=None, d_weights=None,
                             workspace=None, status=None, stream=None, want_d_weights=True):
    """Backward of moe_grouped_ffn (bf16) -> (d_hidden [T,H], d_w13 [E,2I,H], d_w2 [E,H,I], d_weights [T,k] f32)."""
    _dev(hidden, "hidden")
    dt = _dtype_code(hidden)
    T, H = hidden.shape
    E, I2, H2 = w13.shape
    I = I2 // 2
    _dev(w13, "w13", hidden.dtype)
    _dev(w2, "w2", hidden.dtype)
    _dev(d_out, "d_out", hidden.dtype)
    if H2 != H or tuple(w2.shape) != (E, H, I) or tuple(d_out.shape) != (T, H):
        raise ValueError("shape mismatch")
    d = hidden.device
    d_hidden = _out(d_hidden, (T, H), hidden.dtype, d, "d_hidden", stream)
    d_w13 = _out(d_w13, (E, 2 * I, H), hidden.dtype, d, "d_w13", stream)
    d_w2 = _out(d_w2, (E, H, I), hidden.dtype, d, "d_w2", stream)
    if want_d_weights:
        d_weights = _out(d_weights, (T, k), torch.float32, d, "d_weights", stream)
    need = moe_grouped_ffn_backward_workspace_size(dt, T, H, I, E, k)
    if workspace is None:
        workspace = _new(max(need, 1), torch.uint8, d.index, stream)
    _check("moe_grouped_ffn_backward", lib().moe_grouped_ffn_backward(
        _ptr(hidden), _ptr(w13), _ptr(w2), dt, T, H, I, E, k, _ptr(counts), _ptr(offsets),
        _ptr(sorted_token_ids), _ptr(sorted_weights), _ptr(reverse_indices), _ptr(d_out), _ptr(d_hidden),
        _ptr(d_w13), _ptr(d_w2), _ptr(d_weights) if want_d_weights else None, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream, d)))
    return d_hidden, d_w13, d_w2, (d_weights if want_d_weights else None)


def moe_layer_workspace_size(dtype_code, T, H, I, E, k) -> int:
    return int(lib().moe_layer_workspace_size(dtype_code, T, H, I, E, k))


def moe_layer_forward(hidden, router_logits, w13, w2, k, norm_topk_prob=True, out=None,
                      topk_weights=None, topk_indices=None, workspace=None, status=None,
                      stream=None):
    """Whole MoE layer forward -> out [T,H] (hidden's dtype)."""
    _dev(hidden, "hidden")
    _dev(router_logits, "router_logits", torch.float32)
    dt = _dtype_code(hidden)
    T, H = hidden.shape
    E, I2, H2 = w13.shape
    I = I2 // 2
    _dev(w13, "w13", hidden.dtype)
    _dev(w2, "w2", hidden.dtype)
    if H2 != H or tuple(w2.shape) != (E, H, I) or tuple(router_logits.shape) != (T, E):
        raise ValueError("shapes must be hidden [T,H], router_logits [T,E], w13 [E,2I,H], w2 [E,H,I]")
    d = hidden.device
    out = _out(out, (T, H), hidden.dtype, d, "out", stream)
    if topk_weights is not None:
        _out(topk_weights, (T, k), torch.float32, d, "topk_weights", stream)
    if topk_indices is not None:
        _out(topk_indices, (T, k), torch.int32, d, "topk_indices", stream)
    if workspace is None:
        need = moe_layer_workspace_size(dt, T, H, I, E, k)
        workspace = _new(max(need, 1), torch.uint8, d.index, stream)
    _check("moe_layer_forward", lib().moe_layer_forward(
        _ptr(hidden), _ptr(router_logits), _ptr(w13), _ptr(w2), dt, T, H, I, E, k,
        int(bool(norm_topk_prob)), _ptr(out), _ptr(topk_weights), _ptr(topk_indices),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
        _stream(stream, d)))
    return out


_CODES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.float16: MOE_F16}
_ACTIVATIONS = {None: MOE_ACT_NONE, "silu_and_mul": MOE_ACT_SILU_AND_MUL}
_U8, _I32 = torch.uint8, torch.int32


def _code(dtype):
    try:
        return _CODES[dtype]
    except KeyError:
        raise ValueError(f"unsupported dtype {dtype}") from None


# The calls below are made per layer and token, so their checks are few and cheap: one condition per
# tensor, and what was wrong with it is found out afterwards.

def _refuse(t, name, dtype, index):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must be on cuda:{index} (got {t.device})")


def _first(t, name):
    """(address, dtype, device index) of the tensor that the others go by."""
    if not isinstance(t, torch.Tensor):
        _refuse(t, name, None, -1)
    index = t.get_device()
    if index < 0 or not t.is_contiguous():
        _refuse(t, name, None, index)
    if index != _current_device():
        _on_current(index, name)
    return t.data_ptr(), t.dtype, index


def _take(t, name, dtype, index):
    """Address of an input after its checks."""
    try:
        if t.get_device() == index and t.dtype is dtype and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:      # not a tensor
        pass
    _refuse(t, name, dtype, index)


def _give(t, name, shape, dtype, index, stream):
    """(tensor, address) of an output: the caller's after its checks, or a new one."""
    if t is None:
        t = _new(shape, dtype, index, stream)
        return t, t.data_ptr()
    try:
        if t.get_device() == index and t.dtype is dtype and t.is_contiguous() and t.shape == shape:
            return t, t.data_ptr()
    except AttributeError:      # not a tensor
        pass
    _take(t, name, dtype, index)
    raise ValueError(f"{name} must have shape {tuple(shape)}")


def _status_ptr(status, index):
    if status is None:
        return None
    p = _take(status, "status", _I32, index)
    if status.numel() < 1:
        raise ValueError("status must hold an int32 word")
    return p


def _raw(stream, index):
    """Handle of the caller's stream or of the current one, as an integer."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(index)
    return _stream(stream, torch.device("cuda", index)).value


# Workspace sizes follow from the sizes of a call alone, so one that comes again is not asked for again (0.1 us instead
# of 0.8): a 4-bit product that makes its workspace takes the host 13.7 us, and 20.1 where the library is called once to
# say that it needs one.
_sizes = functools.lru_cache(maxsize=4096)


# What follows from the shapes of a call alone is worked out once for each (1 us less a call).
_shapes = functools.lru_cache(maxsize=4096)


def _fits(*sizes):
    """The library's sizes are 32-bit, and ctypes cuts what is larger down to them without a word."""
    if max(sizes) >= 1 << 31:
        raise ValueError(f"sizes must be below 2^31 (got {max(sizes)})")


def _space(workspace, need, index, stream):
    """(tensor, address, bytes) of the caller's workspace, or of a new one where one is needed. The caller holds it
    until the launch; then it goes back to the pool of the call's stream."""
    if workspace is not None:
        return workspace, _take(workspace, "workspace", workspace.dtype, index), workspace.numel() * workspace.element_size()
    if not need:
        return None, None, 0
    workspace = _new(need, _U8, index, stream)
    return workspace, workspace.data_ptr(), need


@_sizes
def moe_grouped_gemm_workspace_size(dtype_code, S, K, N, E) -> int:
    _fits(S, K, N, E)
    return int(lib().moe_grouped_gemm_workspace_size(dtype_code, S, K, N, E))


def moe_grouped_gemm(x, w, offsets, out=None, workspace=None, status=None, stream=None):
    """Rows grouped by expert times the expert's matrix -> y [S, N].

    ``x [S, K]``, ``w [E, N, K]`` (float32, bf16 or float16); ``offsets [E+1]`` int32: expert e owns the
    rows ``offsets[e]`` to ``offsets[e+1] - 1``. Rows without an expert give zero rows."""
    xp, dtype, d = _first(x, "x")
    wp = _take(w, "w", dtype, d)
    op = _take(offsets, "offsets", _I32, d)
    dt = _code(dtype)
    xs, wsh = x.shape, w.shape
    if len(xs) != 2 or len(wsh) != 3 or wsh[2] != xs[1] or offsets.shape != (wsh[0] + 1,):
        raise ValueError("shapes must be x [S, K], w [E, N, K], offsets [E + 1]")
    S, K = xs
    E, N, _ = wsh
    out, yp = _give(out, "out", (S, N), dtype, d, stream)
    space, ws, nb = _space(workspace, moe_grouped_gemm_workspace_size(dt, S, K, N, E), d, stream)
    rc = lib().moe_grouped_gemm(xp, wp, dt, S, K, N, E, op, yp, ws, nb, _status_ptr(status, d), _raw(stream, d))
    if rc:
        _check("moe_grouped_gemm", rc)
    return out


@_sizes
def moe_grouped_gemm_backward_workspace_size(dtype_code, S, K, N, E) -> int:
    _fits(S, K, N, E)
    return int(lib().moe_grouped_gemm_backward_workspace_size(dtype_code, S, K, N, E))


def moe_grouped_gemm_backward(x, w, offsets, d_y, d_x=None, d_w=None, workspace=None, status=None, stream=None,
                              want_d_x=True, want_d_w=True):
    """Gradients of :func:`moe_grouped_gemm` for ``d_y [S, N]`` -> (d_x [S, K], d_w [E, N, K]) in x's dtype.

    One that is not wanted is None. Experts without rows get a zero ``d_w``, rows without an expert a zero ``d_x``."""
    xp, dtype, d = _first(x, "x")
    wp = _take(w, "w", dtype, d)
    gp = _take(d_y, "d_y", dtype, d)
    op = _take(offsets, "offsets", _I32, d)
    dt = _code(dtype)
    xs, wsh = x.shape, w.shape
    if (len(xs) != 2 or len(wsh) != 3 or wsh[2] != xs[1] or offsets.shape != (wsh[0] + 1,)
            or d_y.shape != (xs[0], wsh[1])):
        raise ValueError("shapes must be x [S, K], w [E, N, K], offsets [E + 1], d_y [S, N]")
    S, K = xs
    E, N, _ = wsh
    d_x, dxp = _give(d_x, "d_x", xs, dtype, d, stream) if want_d_x else (None, None)
    d_w, dwp = _give(d_w, "d_w", wsh, dtype, d, stream) if want_d_w else (None, None)
    space, ws, nb = _space(workspace, moe_grouped_gemm_backward_workspace_size(dt, S, K, N, E), d, stream)
    rc = lib().moe_grouped_gemm_backward(xp, wp, gp, dt, S, K, N, E, op, dxp, dwp, ws, nb, _status_ptr(status, d),
                                         _raw(stream, d))
    if rc:
        _check("moe_grouped_gemm_backward", rc)
    return d_x, d_w


@_sizes
def moe_mxfp4_quantize_workspace_size(T, K, with_rows, R) -> int:
    _fits(T, K, R)
    return int(lib().moe_mxfp4_quantize_workspace_size(T, K, int(bool(with_rows)), R))


def moe_mxfp4_quantize(x, rows=None, codes=None, scales=None, workspace=None, status=None, stream=None):
    """4-bit microscaled rows of ``x [T, K]`` (K % 32 == 0) -> (codes [R, K/2] uint8, scales [R, K/32] uint8).

    Blocks of 32 values share the power of two ``2^(scale - 127)``; two codes to a byte, the first one low.
    ``rows [R]`` int32 picks the rows (row r from ``x[rows[r]]``); without it R is T. ``x`` may have more
    than two dimensions when no rows are given: they are kept."""
    xp, dtype, d = _first(x, "x")
    dt = _code(dtype)
    xs = x.shape
    if len(xs) < 2 or xs[-1] % 32:
        raise ValueError("x must be [T, K] (or [..., K] without rows) with K a multiple of 32")
    K = xs[-1]
    if rows is None:
        rp, lead = None, tuple(xs[:-1])
        T = R = xs[:-1].numel()
    else:
        rp = _take(rows, "rows", _I32, d)
        lead = rows.shape
        if len(xs) != 2 or len(lead) != 1:
            raise ValueError("rows must be [R] and x [T, K]")
        T, R = xs[0], lead[0]
    codes, cp = _give(codes, "codes", (*lead, K // 2), _U8, d, stream)
    scales, sp = _give(scales, "scales", (*lead, K // 32), _U8, d, stream)
    space, ws, nb = _space(workspace, moe_mxfp4_quantize_workspace_size(T, K, rp is not None, R), d, stream)
    rc = lib().moe_mxfp4_quantize(xp, dt, T, K, rp, R, cp, sp, ws, nb, _status_ptr(status, d), _raw(stream, d))
    if rc:
        _check("moe_mxfp4_quantize", rc)
    return codes, scales


def moe_mxfp4_dequantize(codes, scales, dtype=torch.bfloat16, out=None, stream=None):
    """The values that ``codes [..., K/2]`` and ``scales [..., K/32]`` stand for -> [..., K] of ``dtype``."""
    cp, _, d = _first(codes, "codes")
    if codes.dtype is not _U8:
        _refuse(codes, "codes", _U8, d)
    sp = _take(scales, "scales", _U8, d)
    dt = _code(dtype)
    cs = codes.shape
    if len(cs) < 1 or cs[-1] % 16:
        raise ValueError("codes must be [..., K / 2] with K a multiple of 32")
    lead, K = cs[:-1], 2 * cs[-1]
    if scales.shape != (*lead, K // 32):
        raise ValueError("shapes must be codes [..., K / 2], scales [..., K / 32]")
    _fits(lead.numel(), K)
    out, op = _give(out, "out", (*lead, K), dtype, d, stream)
    rc = lib().moe_mxfp4_dequantize(cp, sp, lead.numel(), K, dt, op, _raw(stream, d))
    if rc:
        _check("moe_mxfp4_dequantize", rc)
    return out


@_sizes
def moe_mxfp4_grouped_gemm_workspace_size(S, K, N, E, activation=None) -> int:
    _fits(S, K, N, E)
    act = _ACTIVATIONS.get(activation, activation)        # as the product takes it, or the library's code
    return int(lib().moe_mxfp4_grouped_gemm_workspace_size(S, K, N, E, act))


def moe_mxfp4_grouped_gemm(x_codes, x_scales, w_codes, w_scales, offsets, activation=None,
                           out_dtype=torch.bfloat16, out=None, workspace=None, status=None, stream=None):
    """:func:`moe_grouped_gemm` on 4-bit microscaled operands -> y [S, N] of ``out_dtype``.

    ``x_codes [S, K/2]``, ``x_scales [S, K/32]``, ``w_codes [E, N, K/2]``, ``w_scales [E, N, K/32]`` from
    :func:`moe_mxfp4_quantize`. ``activation="silu_and_mul"`` returns [S, N/2]: silu of the first half of
    the columns times the second half."""
    xp, dtype, d = _first(x_codes, "x_codes")
    if dtype is not _U8:
        _refuse(x_codes, "x_codes", _U8, d)
    xsp = _take(x_scales, "x_scales", _U8, d)
    wp = _take(w_codes, "w_codes", _U8, d)
    wsp = _take(w_scales, "w_scales", _U8, d)
    op = _take(offsets, "offsets", _I32, d)
    dt = _code(out_dtype)
    xs, wsh = x_codes.shape, w_codes.shape
    if len(xs) != 2 or len(wsh) != 3:
        raise ValueError("shapes must be x_codes [S, K / 2], w_codes [E, N, K / 2]")
    S, half = xs
    E, N, same = wsh
    if (same != half or half % 16 or x_scales.shape != (S, half // 16) or w_scales.shape != (E, N, half // 16)
            or offsets.shape != (E + 1,)):
        raise ValueError("shapes must be x_codes [S, K / 2], x_scales [S, K / 32], w_codes [E, N, K / 2], "
                         "w_scales [E, N, K / 32], offsets [E + 1] with K a multiple of 32")
    K = 2 * half
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be None or 'silu_and_mul' (got {activation!r})")
    cols, act = N, _ACTIVATIONS[activation]
    if act:
        if N % 2:
            raise ValueError("silu_and_mul needs an even N")
        cols = N // 2
    out, yp = _give(out, "out", (S, cols), out_dtype, d, stream)
    space, ws, nb = _space(workspace, moe_mxfp4_grouped_gemm_workspace_size(S, K, N, E, activation), d, stream)
    rc = lib().moe_mxfp4_grouped_gemm(xp, xsp, wp, wsp, S, K, N, E, op, act, dt, yp, ws, nb, _status_ptr(status, d),
                                      _raw(stream, d))
    if rc:
        _check("moe_mxfp4_grouped_gemm", rc)
    return out


def moe_gather_rows(hidden, sorted_token_ids, offsets, k, out=None, stream=None):
    """Expert-sorted copy of the routed token rows -> x_sorted [T*k, H] (rows p < offsets[E])."""
    _dev(hidden, "hidden")
    dt = _code(hidden.dtype)
    T, H = hidden.shape
    d = hidden.device
    ids = _take(sorted_token_ids, "sorted_token_ids", _I32, d.index)
    offs = _take(offsets, "offsets", _I32, d.index)
    E = offsets.numel() - 1
    _fits(T, H, T * k)
    if sorted_token_ids.numel() < T * k:
        raise ValueError(f"sorted_token_ids must hold T * k = {T * k} ids (got {sorted_token_ids.numel()})")
    out = _out(out, (T * k, H), hidden.dtype, d, "out", stream)
    _check("moe_gather_rows", lib().moe_gather_rows(_ptr(hidden), ids, offs, dt, T, H, E, k, _ptr(out), _stream(stream, d)))
    return out


def moe_ep_receive_index(recv_counts, R, local_counts=None, local_offsets=None, perm=None, workspace=None,
                         stream=None):
    """Owner side of the expert-parallel exchange: recv_counts [G, E_local] int32 (device) ->
    (local_counts [E_local], local_offsets [E_local+1], perm [R]) int32."""
    _dev(recv_counts, "recv_counts", torch.int32)
    G, El = recv_counts.shape
    d = recv_counts.device
    local_counts = _out(local_counts, (El,), torch.int32, d, "local_counts", stream)
    local_offsets = _out(local_offsets, (El + 1,), torch.int32, d, "local_offsets", stream)
    perm = _out(perm, (R,), torch.int32, d, "perm", stream)
    need = int(lib().moe_ep_receive_workspace_size(G, El))
    if workspace is None:
        workspace = _new(max(need, 1), torch.uint8, d.index, stream)
    _check("moe_ep_receive_index", lib().moe_ep_receive_index(
        _ptr(recv_counts), G, El, int(R), _ptr(local_counts), _ptr(local_offsets), _ptr(perm), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream, d)))
    return local_counts, local_offsets, perm


def moe_ep_combine(y_sorted, topk_weights, reverse_indices, offsets, out=None, workspace=None, stream=None):
    """Sender side after the return exchange: out[t] = sum_j w[t,j] * y_sorted[pos(t, j)] -> [T, H]."""
    _dev(y_sorted, "y_sorted")
    dt = _code(y_sorted.dtype)
    d = y_sorted.device
    weights = _take(topk_weights, "topk_weights", _F32, d.index)
    reverse = _take(reverse_indices, "reverse_indices", _I32, d.index)
    offs = _take(offsets, "offsets", _I32, d.index)
    T, k = topk_weights.shape
    H = y_sorted.shape[1]
    E = offsets.numel() - 1
    _fits(T * k, H)
    if y_sorted.shape[0] < T * k or reverse_indices.numel() < T * k:
        raise ValueError(f"y_sorted and reverse_indices must hold T * k = {T * k} rows "
                         f"(got {y_sorted.shape[0]} and {reverse_indices.numel()})")
    out = _out(out, (T, H), y_sorted.dtype, d, "out", stream)
    need = int(lib().moe_ep_combine_workspace_size(T, k))
    if workspace is None:
        workspace = _new(max(need, 1), torch.uint8, d.index, stream)
    _check("moe_ep_combine", lib().moe_ep_combine(
        _ptr(y_sorted), weights, reverse, offs, dt, T, k, H, E, _ptr(out),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream, d)))
    return out


@_sizes
def moe_gather_rows_backward_workspace_size(T, k) -> int:
    _fits(T, k)
    return int(lib().moe_gather_rows_backward_workspace_size(T, k))


@_shapes
def _gather_backward_shape(x, reverse, offsets, k):
    """(T, H, E, shape of d_hidden)"""
    if len(x) != 2 or k < 1 or x[0] % k or reverse != x[:1] or len(offsets) != 1 or offsets[0] < 2:
        raise ValueError("shapes must be d_x_sorted [T * k, H], reverse_indices [T * k], offsets [E + 1]")
    T, H, E = x[0] // k, x[1], offsets[0] - 1
    _fits(x[0], H, E)
    return T, H, E, torch.Size((T, H))


def moe_gather_rows_backward(d_x_sorted, reverse_indices, offsets, k, d_hidden=None, workspace=None, status=None, stream=None):
    """Gradient of :func:`moe_gather_rows`: d_hidden[t] = sum_j d_x_sorted[pos(t, j)] -> [T, H] in d_x_sorted's dtype.

    ``d_x_sorted [T*k, H]`` (float32, bf16 or float16), ``reverse_indices [T*k]`` and ``offsets [E+1]`` from
    :func:`moe_align_by_expert`. Slots without an expert add nothing."""
    xp, dtype, d = _first(d_x_sorted, "d_x_sorted")
    rp = _take(reverse_indices, "reverse_indices", _I32, d)
    op = _take(offsets, "offsets", _I32, d)
    dt = _code(dtype)
    k = int(k)
    T, H, E, shape = _gather_backward_shape(d_x_sorted.shape, reverse_indices.shape, offsets.shape, k)
    d_hidden, hp = _give(d_hidden, "d_hidden", shape, dtype, d, stream)
    space, ws, nb = _space(workspace, moe_gather_rows_backward_workspace_size(T, k), d, stream)
    rc = lib().moe_gather_rows_backward(xp, rp, op, dt, T, H, E, k, hp, ws, nb, _status_ptr(status, d), _raw(stream, d))
    if rc:
        _check("moe_gather_rows_backward", rc)
    return d_hidden


@_sizes
def moe_ep_combine_backward_workspace_size(T, k) -> int:
    _fits(T, k)
    return int(lib().moe_ep_combine_backward_workspace_size(T, k))


@_shapes
def _combine_backward_shape(d_out, y, weights, reverse, offsets):
    """(T, k, H, E, shape of the sorted rows)"""
    if (len(d_out) != 2 or len(weights) != 2 or weights[0] != d_out[0] or reverse != (weights[0] * weights[1],) or len(offsets) != 1
            or offsets[0] < 2 or (y is not None and y != (weights[0] * weights[1], d_out[1]))):
        raise ValueError("shapes must be d_out [T, H], y_sorted [T * k, H], topk_weights [T, k], reverse_indices [T * k], "
                         "offsets [E + 1]")
    (T, H), k, E = d_out, weights[1], offsets[0] - 1
    _fits(T * k, H, E)
    return T, k, H, E, torch.Size((T * k, H))


def moe_ep_combine_backward(d_out, y_sorted, topk_weights, reverse_indices, offsets, d_y=None, d_weights=None, workspace=None,
                            status=None, stream=None, want_d_y=True, want_d_weights=True):
    """Gradients of :func:`moe_ep_combine` for ``d_out [T, H]`` -> (d_y [T*k, H] in d_out's dtype, d_weights [T, k] float32).

    One that is not wanted is None (``y_sorted`` is read for ``d_weights`` only and may be None without). Slots without
    an expert have ``d_weights`` 0; rows of ``d_y`` behind the last expert's are left as they are."""
    gp, dtype, d = _first(d_out, "d_out")
    yp = _take(y_sorted, "y_sorted", dtype, d) if y_sorted is not None or want_d_weights else None
    wp = _take(topk_weights, "topk_weights", torch.float32, d)
    rp = _take(reverse_indices, "reverse_indices", _I32, d)
    op = _take(offsets, "offsets", _I32, d)
    dt = _code(dtype)
    T, k, H, E, rows = _combine_backward_shape(d_out.shape, None if y_sorted is None else y_sorted.shape, topk_weights.shape,
                                               reverse_indices.shape, offsets.shape)
    d_y, dyp = _give(d_y, "d_y", rows, dtype, d, stream) if want_d_y else (None, None)
    d_weights, dwp = _give(d_weights, "d_weights", topk_weights.shape, torch.float32, d, stream) if want_d_weights else (None, None)
    space, ws, nb = _space(workspace, moe_ep_combine_backward_workspace_size(T, k), d, stream)
    rc = lib().moe_ep_combine_backward(gp, yp, wp, rp, op, dt, T, k, H, E, dyp, dwp, ws, nb, _status_ptr(status, d), _raw(stream, d))
    if rc:
        _check("moe_ep_combine_backward", rc)
    return d_y, d_weights


_F8 = torch.float8_e4m3fn
_F32 = torch.float32
FP8_BLOCK = 128


def _pieces(n):
    return -(-n // FP8_BLOCK)


@_shapes
def _fp8_shape(shape, block_rows, name):
    """(matrices, rows, columns, shape of the scales) of values [..., K], or of matrices [..., N, K] with 128 x 128 blocks."""
    if block_rows not in (1, FP8_BLOCK):
        raise ValueError(f"block_rows must be 1 or {FP8_BLOCK} (got {block_rows})")
    if len(shape) < (1 if block_rows == 1 else 2) or shape[-1] % 16:
        raise ValueError(f"{name} must be [..., K] ([..., N, K] with block_rows {FP8_BLOCK}) with K a multiple of 16")
    K = shape[-1]
    if block_rows == 1:
        M, N, scales = 1, shape[:-1].numel(), torch.Size((*shape[:-1], _pieces(K)))
    else:
        M, N = shape[:-2].numel(), shape[-2]
        scales = torch.Size((*shape[:-2], _pieces(N), _pieces(K)))
    _fits(M, N, K, M * N)
    return M, N, K, scales


def moe_fp8_quantize(x, block_rows=1, codes=None, scales=None, stream=None):
    """8-bit values of ``x`` with a float32 scale per block -> (codes float8_e4m3fn as x, scales).

    ``block_rows=1``: ``x [..., K]`` and a scale for each 128 values of a row, ``scales [..., ceil(K/128)]`` (activations).
    ``block_rows=128``: ``x [..., N, K]`` and a scale for 128 x 128 values, ``[..., ceil(N/128), ceil(K/128)]`` (weights).
    K must be a multiple of 16."""
    xp, dtype, d = _first(x, "x")
    dt = _code(dtype)
    M, N, K, ss = _fp8_shape(x.shape, block_rows, "x")
    codes, cp = _give(codes, "codes", x.shape, _F8, d, stream)
    scales, sp = _give(scales, "scales", ss, _F32, d, stream)
    rc = lib().moe_fp8_quantize(xp, dt, M, N, K, block_rows, cp, sp, _raw(stream, d))
    if rc:
        _check("moe_fp8_quantize", rc)
    return codes, scales


def moe_fp8_dequantize(codes, scales, dtype=torch.bfloat16, block_rows=1, out=None, stream=None):
    """The values that ``codes`` and ``scales`` of :func:`moe_fp8_quantize` stand for, in ``dtype``."""
    cp, _, d = _first(codes, "codes")
    if codes.dtype is not _F8:
        _refuse(codes, "codes", _F8, d)
    sp = _take(scales, "scales", _F32, d)
    dt = _code(dtype)
    M, N, K, ss = _fp8_shape(codes.shape, block_rows, "codes")
    if scales.shape != ss:
        raise ValueError(f"scales must have shape {tuple(ss)}")
    out, op = _give(out, "out", codes.shape, dtype, d, stream)
    rc = lib().moe_fp8_dequantize(cp, sp, M, N, K, block_rows, dt, op, _raw(stream, d))
    if rc:
        _check("moe_fp8_dequantize", rc)
    return out


def moe_rms_norm_fp8(x, weight, residual=None, eps=1e-6, want_normed=False, codes=None, scales=None, residual_out=None, normed=None,
                     stream=None):
    """Addition of the residual and root-mean-square norm, as 8-bit rows -> (codes, scales, residual_out, normed).

    h = x + residual (rounded to x's dtype); n = h / sqrt(mean h^2 + eps) * weight in float32; ``codes`` and ``scales``
    hold n as :func:`moe_fp8_quantize` does, ``residual_out`` h (None without a residual; pass the residual itself to
    update it in place), ``normed`` n in x's dtype (None unless wanted or given). ``x``, ``residual [..., H]``,
    ``weight [H]`` of one dtype, H a multiple of 16."""
    xp, dtype, d = _first(x, "x")
    wp = _take(weight, "weight", dtype, d)
    rp = None if residual is None else _take(residual, "residual", dtype, d)
    dt = _code(dtype)
    xs = x.shape
    _, T, H, ss = _fp8_shape(xs, 1, "x")
    if weight.shape != xs[-1:] or (residual is not None and residual.shape != xs):
        raise ValueError("shapes must be x [..., H], weight [H], residual as x")
    if residual is None and residual_out is not None:
        raise ValueError("residual_out needs a residual")
    codes, cp = _give(codes, "codes", xs, _F8, d, stream)
    scales, sp = _give(scales, "scales", ss, _F32, d, stream)
    residual_out, op = (None, None) if residual is None else _give(residual_out, "residual_out", xs, dtype, d, stream)
    normed, np_ = _give(normed, "normed", xs, dtype, d, stream) if want_normed or normed is not None else (None, None)
    rc = lib().moe_rms_norm_fp8(xp, rp, wp, dt, T, H, eps, cp, sp, op, np_, _raw(stream, d))
    if rc:
        _check("moe_rms_norm_fp8", rc)
    return codes, scales, residual_out, normed


@_shapes
def _fp8_gather_shape(codes, scales, ids, offsets):
    """(T, H, S, E, shapes of the outputs)"""
    if (len(codes) != 2 or codes[1] % 16 or scales != (codes[0], _pieces(codes[1])) or len(ids) != 1 or len(offsets) != 1
            or offsets[0] < 2):
        raise ValueError("shapes must be codes [T, H], scales [T, ceil(H / 128)], sorted_token_ids [S], offsets [E + 1] with H a "
                         "multiple of 16")
    (T, H), S, E = codes, ids[0], offsets[0] - 1
    _fits(T, H, S, E)
    return T, H, S, E, torch.Size((S, H)), torch.Size((S, _pieces(H)))


def moe_fp8_gather_rows(codes, scales, sorted_token_ids, offsets, out=None, out_scales=None, status=None, stream=None):
    """Expert-sorted copies of 8-bit rows -> (codes [S, H], scales [S, ceil(H/128)]), rows p < offsets[E].

    ``codes [T, H]``, ``scales [T, ceil(H/128)]``; ``sorted_token_ids [S]`` and ``offsets [E+1]`` from
    :func:`moe_align_by_expert`. Rows behind the last expert's are left as they are."""
    cp, dtype, d = _first(codes, "codes")
    if dtype is not _F8:
        _refuse(codes, "codes", _F8, d)
    sp = _take(scales, "scales", _F32, d)
    ip = _take(sorted_token_ids, "sorted_token_ids", _I32, d)
    op = _take(offsets, "offsets", _I32, d)
    T, H, S, E, rows, row_scales = _fp8_gather_shape(codes.shape, scales.shape, sorted_token_ids.shape, offsets.shape)
    out, xp = _give(out, "out", rows, _F8, d, stream)
    out_scales, xsp = _give(out_scales, "out_scales", row_scales, _F32, d, stream)
    rc = lib().moe_fp8_gather_rows(cp, sp, ip, op, T, H, E, S, xp, xsp, _status_ptr(status, d), _raw(stream, d))
    if rc:
        _check("moe_fp8_gather_rows", rc)
    return out, out_scales


@_shapes
def _fp8_product_shape(x, x_scales, w, w_scales, offsets, activation):
    """(S, K, N, E, the activation's code, shape of y)"""
    if (len(x) != 2 or len(w) != 3 or w[2] != x[1] or x[1] % 16 or x_scales != (x[0], _pieces(x[1]))
            or w_scales != (w[0], _pieces(w[1]), _pieces(w[2])) or offsets != (w[0] + 1,)):
        raise ValueError("shapes must be x_codes [S, K], x_scales [S, ceil(K / 128)], w_codes [E, N, K], "
                         "w_scales [E, ceil(N / 128), ceil(K / 128)], offsets [E + 1] with K a multiple of 16")
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be None or 'silu_and_mul' (got {activation!r})")
    (S, K), (E, N, _), act = x, w, _ACTIVATIONS[activation]
    if act and N % 32:
        raise ValueError("silu_and_mul needs N to be a multiple of 32")
    _fits(S, K, N, E)
    return S, K, N, E, act, torch.Size((S, N // 2 if act else N))


def moe_fp8_grouped_gemm(x_codes, x_scales, w_codes, w_scales, offsets, activation=None, out_dtype=torch.bfloat16, out=None,
                         status=None, stream=None):
    """:func:`moe_grouped_gemm` on 8-bit operands -> y [S, N] of ``out_dtype``.

    ``x_codes [S, K]`` with ``x_scales [S, ceil(K/128)]``, ``w_codes [E, N, K]`` with
    ``w_scales [E, ceil(N/128), ceil(K/128)]`` as :func:`moe_fp8_quantize` makes them (``block_rows`` 1 and 128), K a
    multiple of 16. ``activation="silu_and_mul"`` returns [S, N/2]: silu of the first half of the columns times the
    second half (N a multiple of 32); its exponential and division are the fast ones for float32 results, too."""
    xp, dtype, d = _first(x_codes, "x_codes")
    if dtype is not _F8:
        _refuse(x_codes, "x_codes", _F8, d)
    xsp = _take(x_scales, "x_scales", _F32, d)
    wp = _take(w_codes, "w_codes", _F8, d)
    wsp = _take(w_scales, "w_scales", _F32, d)
    op = _take(offsets, "offsets", _I32, d)
    dt = _code(out_dtype)
    S, K, N, E, act, shape = _fp8_product_shape(x_codes.shape, x_scales.shape, w_codes.shape, w_scales.shape, offsets.shape, activation)
    out, yp = _give(out, "out", shape, out_dtype, d, stream)
    rc = lib().moe_fp8_grouped_gemm(xp, xsp, wp, wsp, S, K, N, E, op, act, dt, yp, _status_ptr(status, d), _raw(stream, d))
    if rc:
        _check("moe_fp8_grouped_gemm", rc)
    return out


def set_wait_limit_ns(ns: int) -> int:
    """Limit of the waits of the tensor-core kernels (FFN, grouped, 4-bit and 8-bit products) on their other roles (0: the
    default, 2 s); returns the previous limit."""
    return int(lib().moe_set_wait_limit_ns(int(ns)))


def profiler_enable(on: bool = True) -> None:
    lib().moe_profiler_enable(int(bool(on)))


def profiler_report() -> dict:
    """Per-kernel {"launches": n, "total_ms": t} since the last report (synchronises)."""
    buf = ctypes.create_string_buffer(1 << 20)
    n = lib().moe_profiler_report(buf, len(buf))
    if n >= len(buf):
        raise RuntimeError("profiler report truncated")
    return json.loads(buf.value.decode())
