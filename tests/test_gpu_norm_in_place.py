"""The norm with its outputs over its inputs, in three types, at widths of every kernel: the results of a call with memory of
their own."""
import pytest
import torch

from gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,H", [(5, 128), (70, 512), (33, 1024), (6, 2064), (3, 4112), (900, 8192), (400, 8208), (7, 20000)])
def test_outputs_over_inputs(dtype, T, H):
    moe = need_gpu()
    g = torch.Generator(device=DEV).manual_seed(H)
    x, r = (torch.randn(T, H, generator=g, device=DEV).to(dtype) for _ in range(2))
    w = torch.rand(H, generator=g, device=DEV).to(dtype)
    call = lambda x, **kw: moe.moe_rms_norm_fp8(x, w, **kw)  # noqa: E731

    def same(got, want):
        assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(got[1], want[1])
        assert all(a is None or b is None or torch.equal(a, b) for a, b in zip(got[2:], want[2:]))

    want = call(x, residual=r, want_normed=True)
    alone = call(x, want_normed=True)
    assert torch.equal(want[2], (x.float() + r.float()).to(dtype))
    for _ in range(3):
        x2, r2 = x.clone(), r.clone()
        same(call(x2, residual=r2, residual_out=r2, normed=x2), want)
        assert torch.equal(r2, want[2]) and torch.equal(x2, want[3])
        x2 = x.clone()
        same(call(x2, residual=r, residual_out=x2, want_normed=True), want)
        assert torch.equal(x2, want[2])
        x2 = x.clone()
        same(call(x2, normed=x2), alone)
        assert torch.equal(x2, alone[3])
