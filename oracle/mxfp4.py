"""4-bit microscaled values in float64: blocks of 32, a power-of-two scale, e2m1 codes.

The code of a value is found by its distances to all eight magnitudes, the scale by
searching the exponent, so nothing here shares a step with a bit-level implementation.
"""
import numpy as np

BLOCK = 32
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
NAN_SCALE = 255


def quantize(x):
    """x [..., K] -> (codes [..., K] uint8 in 0..15, scales [..., K/32] uint8)."""
    x = np.asarray(x, np.float64)
    v = x.reshape(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)
    fine = np.isfinite(v).all(-1)
    most = np.where(fine, np.abs(v).max(-1), 0.0)
    s = np.full(most.shape, -127)
    for e in range(-125, 128):                      # floor(log2 most) >= e, by comparison with the powers themselves
        s = np.where(most >= 2.0 ** e, np.maximum(e - 2, -127), s)
    a = np.where(fine[..., None], v, 0.0) / (2.0 ** s.astype(np.float64))[..., None]
    mag = np.minimum(np.abs(a), 6.0)
    dist = np.abs(mag[..., None] - GRID)
    best = dist.min(-1, keepdims=True)
    near = dist == best                              # two entries at a tie: take the even index
    even = np.arange(8) % 2 == 0
    tie = near.sum(-1) == 2
    code = np.where(tie, (near & even).argmax(-1), near.argmax(-1))
    code = (code + 8 * (np.signbit(v) & fine[..., None])).astype(np.uint8)
    scale = np.where(fine, s + 127, NAN_SCALE).astype(np.uint8)
    return code.reshape(x.shape), scale


def pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    out = np.empty(packed.shape[:-1] + (2 * packed.shape[-1],), np.uint8)
    out[..., 0::2], out[..., 1::2] = packed & 15, packed >> 4
    return out


def dequantize(code, scale):
    """Values of codes (one per value) under their scales."""
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    power = np.where(scale == NAN_SCALE, np.nan, 2.0 ** (scale.astype(np.float64) - 127))
    return (v.reshape(*scale.shape, BLOCK) * power[..., None]).reshape(code.shape)


def silu_and_mul(y):
    half = y.shape[-1] // 2
    g, u = y[..., :half], y[..., half:]
    return g / (1.0 + np.exp(-g)) * u
