"""8-bit values (e4m3) with a float32 scale per block of 128 values of a row, or of 128 x 128 of a matrix.

The code of a value is found by its distances to all 127 magnitudes; scales, their inverses and the scaled values are
float32, each step rounded once, as the format says. What the codes stand for, products and norms are in float64.
"""
import numpy as np

BLOCK = 128
NAN_CODE = 0x7F
_C = np.arange(127)
# code c: exponent c >> 3 (bias 7), mantissa c & 7; no infinities
GRID = np.where(_C < 8, _C * 2.0 ** -9, (8 + (_C & 7)) * 2.0 ** ((_C >> 3) - 10.0))


def pieces(n):
    return -(-n // BLOCK)


def _spread(scales, shape, block_rows):
    """Scales as they apply to single values of `shape`."""
    s = np.repeat(scales, BLOCK, axis=-1)[..., : shape[-1]]
    return np.repeat(s, BLOCK, axis=-2)[..., : shape[-2], :] if block_rows > 1 else s


def encode(v):
    """Nearest codes of float values (ties to the even code, magnitudes above 448 to 448)."""
    v = np.asarray(v, np.float64)
    mag = np.minimum(np.abs(v), GRID[-1]).reshape(-1)
    code = np.empty(mag.shape, np.uint8)
    for i in range(0, mag.size, 1 << 14):
        d = np.abs(mag[i:i + (1 << 14), None] - GRID)
        near = d == d.min(1, keepdims=True)
        even = near & (_C % 2 == 0)
        code[i:i + (1 << 14)] = np.where(near.sum(1) == 2, even.argmax(1), near.argmax(1))
    return (code.reshape(v.shape) + 128 * np.signbit(v)).astype(np.uint8)


def quantize(x, block_rows=1):
    """x [..., K] (float32 values) -> (codes uint8 as x, scales float32)."""
    x = np.asarray(x, np.float32)
    K = x.shape[-1]
    rows = x.shape[-2] if block_rows > 1 else 0
    pad = [(0, 0)] * x.ndim
    pad[-1] = (0, pieces(K) * BLOCK - K)
    if block_rows > 1:
        pad[-2] = (0, pieces(rows) * BLOCK - rows)
    a = np.pad(np.abs(x), pad)
    a = a.reshape(*a.shape[:-1], pieces(K), BLOCK)
    with np.errstate(invalid="ignore"):
        most = a.max(-1)                                   # NaN stays NaN
        if block_rows > 1:
            most = most.reshape(*most.shape[:-2], pieces(rows), BLOCK, most.shape[-1]).max(-2)
        fine = np.isfinite(most)
        scales = np.maximum(np.where(fine, most, 0).astype(np.float32) / np.float32(448), np.float32(2.0 ** -126))
        inv = np.float32(1) / scales
        f = _spread(fine, x.shape, block_rows)
        scaled = np.where(f, x, 0) * _spread(inv, x.shape, block_rows)
    codes = np.where(f, encode(scaled), 0).astype(np.uint8)
    return codes, np.where(fine, scales, np.float32(np.nan)).astype(np.float32)


def decode(codes):
    c = codes & 127
    v = np.where(c == NAN_CODE, np.nan, GRID[np.minimum(c, 126)])
    return np.where(codes & 128, -v, v)


def dequantize(codes, scales, block_rows=1):
    """What codes stand for under their scales, in float64."""
    return decode(codes) * _spread(scales.astype(np.float64), codes.shape, block_rows)


def rms_norm(h, weight, eps):
    """h * (1 / sqrt(mean h^2 + eps)) * weight in float64 (h: the sum with the residual, as the stream holds it)."""
    h = np.asarray(h, np.float64)
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
