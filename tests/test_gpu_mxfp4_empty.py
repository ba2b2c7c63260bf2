"""Quantisation of rows of a matrix that has none: every row wanted is zero and reported, however many there are."""
import pytest
import torch

from gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R", [1, 2, 2047, 2048, 2049, 70000])      # from 2048 rows of 2048 on a matrix with rows takes two kernels
def test_rows_of_an_empty_matrix(R):
    moe = need_gpu()
    x = torch.empty(0, 2048, dtype=torch.bfloat16, device=DEV)
    rows = torch.zeros(R, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    codes = torch.full((R, 1024), 7, dtype=torch.uint8, device=DEV)
    scales = torch.full((R, 64), 7, dtype=torch.uint8, device=DEV)
    moe.moe_mxfp4_quantize(x, rows=rows, codes=codes, scales=scales, status=status)
    assert not codes.any() and not scales.any()
    assert int(status.item()) == moe.MOE_STATUS_BAD_INDEX
    good = torch.randn(4, 64, device=DEV)                          # the next call is not told of an earlier one's error
    assert torch.equal(moe.moe_mxfp4_quantize(good)[0], moe.moe_mxfp4_quantize(good, rows=torch.arange(4, dtype=torch.int32, device=DEV))[0])
