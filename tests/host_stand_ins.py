"""The binding without a GPU: tensors in host memory that say they lie on one, and a library that answers every call
with 0 and every workspace size with 512."""
import torch

import mixture_experts_routing_token_gb300._binding as binding

I, F, B, U = torch.int32, torch.float32, torch.bfloat16, torch.uint8
T, K, E, H, M = 6, 2, 4, 64, 32      # tokens, experts a token, experts, hidden and intermediate width


class OnGpu(torch.Tensor):
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 0))

    def get_device(self):
        return 0


class Lib:
    def __init__(self):
        self.called = []

    def __getattr__(self, name):
        if not name.endswith("_size"):
            self.called.append(name)
        return lambda *args: 512 if name.endswith("_size") else 0


def gpu(*shape, dtype=F, device=None):
    return torch.zeros(shape, dtype=dtype, device=device).as_subclass(OnGpu)


def forget_sizes():
    for f in vars(binding).values():
        if hasattr(f, "cache_clear") and f.__name__.endswith("_size"):
            f.cache_clear()


def aligned():
    return (gpu(E, dtype=I), gpu(E + 1, dtype=I), gpu(T * K, dtype=I), gpu(T * K), gpu(T * K, dtype=I))


def ffn():
    return gpu(T, H, dtype=B), gpu(E, 2 * M, H, dtype=B), gpu(E, H, M, dtype=B)


def codes(*shape):
    return gpu(*shape[:-1], shape[-1] // 2, dtype=U), gpu(*shape[:-1], shape[-1] // 32, dtype=U)


# every call that takes tensors, on the stream `s`
CALLS = {
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
    "product": lambda s: binding.moe_grouped_gemm(gpu(T, H), gpu(E, M, H), gpu(E + 1, dtype=I), stream=s),
    "gradients": lambda s: binding.moe_grouped_gemm_backward(gpu(T, H), gpu(E, M, H), gpu(E + 1, dtype=I), gpu(T, M), stream=s),
    "quantize": lambda s: binding.moe_mxfp4_quantize(gpu(T, H), rows=gpu(T, dtype=I), stream=s),
    "dequantize": lambda s: binding.moe_mxfp4_dequantize(*codes(T, H), stream=s),
    "product4": lambda s: binding.moe_mxfp4_grouped_gemm(*codes(T, H), *codes(E, M, H), gpu(E + 1, dtype=I), stream=s),
}
