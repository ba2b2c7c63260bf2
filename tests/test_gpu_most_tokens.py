"""As many tokens as an int holds, on the calls whose launches count CTAs from them."""
import pytest
import torch

from gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


@pytest.fixture(autouse=True)
def room():
    """These calls need up to 120 GB; other tests' blocks go back first, and these ones' afterwards."""
    need_gpu()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 160 << 30:
        pytest.skip("less than 160 GB free")
    yield
    torch.cuda.empty_cache()


def test_gradients_of_one_row_a_token():
    moe = need_gpu()
    g = torch.Generator(device=DEV).manual_seed(0)
    reverse = torch.arange(MOST - 1, -1, -1, dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 5, MOST], dtype=torch.int32, device=DEV)
    rows = torch.empty(MOST, 1, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    d_hidden = moe.moe_gather_rows_backward(rows, reverse, off, 1)
    assert torch.equal(d_hidden.flip(0), rows)            # one row each: a copy
    del d_hidden
    ones = torch.ones(MOST, 1, device=DEV)
    d_y, d_w = moe.moe_ep_combine_backward(rows, torch.ones_like(rows), ones, reverse, off)
    assert torch.equal(d_y.flip(0), rows) and torch.equal(d_w, rows.float())
    del d_y, d_w
    assert torch.equal(moe.moe_ep_combine(rows, ones, reverse, off).flip(0), rows)
    assert torch.equal(moe.moe_gather_rows(rows, reverse, off, 1).flip(0), rows)


def test_norm_of_the_narrowest_rows():
    moe = need_gpu()
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty(MOST, 16, dtype=torch.bfloat16, device=DEV)
    ends = [slice(0, 1000), slice(MOST // 2, MOST // 2 + 1000), slice(MOST - 1000, MOST)]
    for s in ends:
        x[s] = torch.randn(1000, 16, generator=g, device=DEV)
    w = torch.rand(16, generator=g, device=DEV).to(torch.bfloat16)
    codes, scales, _, _ = moe.moe_rms_norm_fp8(x, w)
    for s in ends:
        want = moe.moe_rms_norm_fp8(x[s].contiguous(), w)
        assert torch.equal(codes[s].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(scales[s], want[1])
