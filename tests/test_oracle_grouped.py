"""The oracle of the grouped products and of the 4-bit microscaled values, against hand-worked
cases, brute force and differences (no GPU)."""
import numpy as np
import pytest

from oracle import grouped, mxfp4


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def test_product_row_by_row():
    rng = np.random.default_rng(0)
    off = offsets_of([3, 0, 2, 1])
    x, w = rng.standard_normal((8, 5)), rng.standard_normal((4, 3, 5))     # two rows beyond the groups
    y = grouped.grouped_gemm(x, w, off)
    e = grouped.expert_of_rows(off, 8)
    assert e.tolist() == [0, 0, 0, 2, 2, 3, -1, -1]
    for p in range(8):
        want = np.zeros(3) if e[p] < 0 else np.array([sum(x[p, k] * w[e[p], n, k] for k in range(5)) for n in range(3)])
        np.testing.assert_allclose(y[p], want, rtol=1e-13, atol=1e-13)


def test_gradient_by_differences():
    rng = np.random.default_rng(1)
    off = offsets_of([2, 0, 3])
    x, w, d_y = rng.standard_normal((6, 4)), rng.standard_normal((3, 3, 4)), rng.standard_normal((6, 3))
    d_x, d_w = grouped.grouped_gemm_backward(x, w, off, d_y)
    f = lambda x, w: float((grouped.grouped_gemm(x, w, off) * d_y).sum())  # noqa: E731
    for arr, grad in ((x, d_x), (w, d_w)):
        for i in np.ndindex(arr.shape):
            keep = arr[i]
            arr[i] = keep + 1e-4
            up = f(x, w)
            arr[i] = keep - 1e-4
            down = f(x, w)
            arr[i] = keep
            assert abs((up - down) / 2e-4 - grad[i]) < 1e-9     # the function is linear in each entry
    assert not d_x[5].any() and not d_w[1].any()


def test_quantize_hand_worked():
    x = np.zeros((1, 32))
    x[0, :12] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -5.0, 7.9, -0.2, 0.26, 6.1]
    code, scale = mxfp4.quantize(x)                  # largest 7.9: floor(log2) = 2, so the scale is 1
    assert scale.tolist() == [[127]]
    assert code[0, :12].tolist() == [6, 0, 2, 2, 4, 4, 6, 14, 7, 8, 1, 7]
    v = mxfp4.dequantize(code, scale)
    assert v[0, :12].tolist() == [4.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, -4.0, 6.0, 0.0, 0.5, 6.0]


@pytest.mark.parametrize("e", [-149, -140, -126, -125, -124, -1, 0, 1, 126, 127])
def test_quantize_powers_of_two(e):
    x = np.zeros((1, 32))
    x[0, 3] = 2.0 ** e
    code, scale = mxfp4.quantize(x)
    assert scale[0, 0] == max(e - 2, -127) + 127
    want = 2.0 ** e if e >= -127 - 1 else 0.0        # half the smallest scale is the smallest value held
    assert mxfp4.dequantize(code, scale)[0, 3] == want


def test_quantize_nonfinite_and_zero_blocks():
    x = np.ones((1, 128))
    x[0, 5], x[0, 40], x[0, 64:96] = np.nan, -np.inf, 0.0
    code, scale = mxfp4.quantize(x)
    assert scale.tolist() == [[255, 255, 0, 125]]
    assert not code[0, :96].any()
    v = mxfp4.dequantize(code, scale)
    assert np.isnan(v[0, :64]).all() and not v[0, 64:96].any() and (v[0, 96:] == 1.0).all()


def test_pack_round_trip():
    code = np.random.default_rng(2).integers(0, 16, (3, 64)).astype(np.uint8)
    packed = mxfp4.pack(code)
    assert packed[0, 0] == code[0, 0] + 16 * code[0, 1]
    assert (mxfp4.unpack(packed) == code).all()


def test_quantization_error_bound():
    # between 4 and 8 (in units of the scale) the grid has 4 and 6: the largest relative error of the
    # block's largest value is at 8-: 2 / 8
    x = np.random.default_rng(3).standard_normal((200, 64))
    v = mxfp4.dequantize(*mxfp4.quantize(x))
    most = np.abs(x).reshape(200, 2, 32).max(-1, keepdims=True)
    assert (np.abs(v - x).reshape(200, 2, 32) <= most / 4).all()
