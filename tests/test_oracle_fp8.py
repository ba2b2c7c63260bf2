"""The oracles of the 8-bit values and of the gradients of sorted rows, against hand-worked cases and differences (no GPU)."""
import numpy as np
import pytest
import torch

from oracle import fp8, sorted_rows


def test_grid():
    assert fp8.GRID[1] == 2.0 ** -9 and fp8.GRID[8] == 2.0 ** -6 and fp8.GRID[0x38] == 1.0 and fp8.GRID[126] == 448
    assert (np.diff(fp8.GRID) > 0).all()


def test_encode_hand_worked():
    v = np.array([0.0, -0.0, 1.0, 1.0625, 1.1875, 448, 460, 1e9, -2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0])
    # 1.0625 lies between 1 (0x38) and 1.125 (0x39), 1.1875 between 0x39 and 0x3a; 2^-10 between 0 and 2^-9; 17 between 16 and 18
    want = [0, 0x80, 0x38, 0x38, 0x3A, 0x7E, 0x7E, 0x7E, 0x81, 0, 2, 0x58, 0x5A]
    assert fp8.encode(v).tolist() == want


def test_encode_is_torchs_rounding():
    x = torch.randn(4000, generator=torch.Generator().manual_seed(0)) * torch.exp2(torch.randint(-12, 8, (4000,)).float())
    x = x.clamp(-448, 448)
    assert (fp8.encode(x.numpy()) == x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()).all()


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("N,K", [(1, 16), (3, 128), (130, 272), (128, 256), (200, 400)])
def test_quantize_blocks(block_rows, N, K):
    x = np.random.default_rng(N).standard_normal((2, N, K)).astype(np.float32)
    codes, scales = fp8.quantize(x, block_rows)
    v = fp8.dequantize(codes, scales, block_rows)
    assert scales.shape == (2, N if block_rows == 1 else fp8.pieces(N), fp8.pieces(K))
    for m in range(2):
        for r0 in range(0, N, block_rows):
            for c0 in range(0, K, 128):
                b = x[m, r0:r0 + block_rows, c0:c0 + 128]
                s = scales[m, r0 // block_rows, c0 // 128]
                assert s == np.float32(np.abs(b).max()) / np.float32(448)
                # off by half a step: 2^-4 of the value, or of the smallest normal one (2^-6)
                got = v[m, r0:r0 + block_rows, c0:c0 + 128]
                assert (np.abs(got - b) <= (1 + 1e-6) * np.maximum(np.abs(b) / 16, float(s) * 2.0 ** -10)).all()


def test_quantize_zero_small_and_nonfinite_blocks():
    x = np.zeros((1, 640), np.float32)
    x[0, 128], x[0, 256], x[0, 300], x[0, 390], x[0, 512:] = 1e-40, np.inf, 1.0, np.nan, 448.0
    codes, scales = fp8.quantize(x)
    assert scales[0, :2].tolist() == [2.0 ** -126] * 2 and np.isnan(scales[0, 2:4]).all() and scales[0, 4] == 1
    assert not codes[0, :128].any() and not codes[0, 256:512].any() and (codes[0, 512:] == 0x7E).all()
    assert abs(fp8.dequantize(codes, scales)[0, 128] - 1e-40) <= 2.0 ** -136
    assert np.isnan(fp8.dequantize(codes, scales)[0, 256:512]).all()


def test_norm_by_hand():
    n = fp8.rms_norm([[3.0, 4.0, 0.0, 0.0]], [1, 2, 1, 1], 0.0)
    np.testing.assert_allclose(n, [[1.2, 3.2, 0, 0]], rtol=1e-15)


def routing(T, k, dropped, seed=0):
    rng = np.random.default_rng(seed)
    reverse = rng.permutation(T * k).astype(np.int32)
    return reverse, T * k - dropped, rng


def test_gradients_of_sorted_rows_by_differences():
    T, k, H = 4, 3, 5
    reverse, n, rng = routing(T, k, 2)
    hidden, d_x = rng.standard_normal((T, H)), rng.standard_normal((T * k, H))
    y, w, d_out = rng.standard_normal((T * k, H)), rng.standard_normal((T, k)), rng.standard_normal((T, H))
    d_y, d_w = sorted_rows.combine_backward(d_out, y, w, reverse, n)
    cases = [(lambda: float((sorted_rows.gather(hidden, reverse, n, k) * d_x[:n]).sum()), hidden,
              sorted_rows.gather_backward(d_x, reverse, n, T, k)),
             (lambda: float((sorted_rows.combine(y, w, reverse, n) * d_out).sum()), y, np.concatenate([d_y, np.zeros((2, H))])),
             (lambda: float((sorted_rows.combine(y, w, reverse, n) * d_out).sum()), w, d_w)]
    for f, arr, grad in cases:
        for i in np.ndindex(arr.shape):
            keep = arr[i]
            arr[i] = keep + 1e-4
            up = f()
            arr[i] = keep - 1e-4
            down = f()
            arr[i] = keep
            assert abs((up - down) / 2e-4 - grad[i]) < 1e-9     # linear in each entry
