"""MX4 in float64, by its definition (test infrastructure only).

A block of 32 consecutive elements of a row shares the scale 2^s, s =
max(floor(log2(max |x|)) - 2, -127); an element's code is the E2M1 level
nearest to x / 2^s, ties to the even code, clipped to the largest.  A block
with a NaN or an infinity has the scale byte 255 and zero codes.
"""

import numpy as np

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)


def quantize(x):
    """x [rows, cols] (cols % 32 == 0, values exact in float64) -> codes uint8
    [rows, cols] (bit 3 the sign) and scale bytes uint8 [rows, cols / 32]."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    b = x.reshape(rows, cols // 32, 32)
    bad = ~np.isfinite(b).all(2)
    top = np.where(np.isfinite(b), np.abs(b), 0.0).max(2)
    # frexp: top = m 2^e with m in [0.5, 1), so floor(log2 top) = e - 1
    s = np.maximum(np.where(top > 0, np.frexp(top)[1] - 1, -1000) - 2, -127)
    with np.errstate(invalid="ignore"):
        m = np.abs(b) / np.exp2(s.astype(np.float64))[:, :, None]
    m = np.where(np.isfinite(m), m, 0.0)
    dist = np.abs(m[..., None] - LEVELS)
    best = dist.min(-1, keepdims=True)
    near = dist == best
    k = np.arange(8)
    # the even code of two equally near ones
    code = np.where(near, np.where(k % 2 == 0, k, k + 100), 1000).min(-1) % 100
    code = code + 8 * np.signbit(b)
    code = np.where(bad[:, :, None], 0, code).astype(np.uint8).reshape(rows, cols)
    return code, np.where(bad, 255, s + 127).astype(np.uint8)


def values(codes, scale_bytes):
    """float64 values of codes [rows, cols] and scale bytes [rows, cols / 32]."""
    v = LEVELS[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    f = np.where(scale_bytes == 255, np.nan, np.exp2(scale_bytes.astype(np.float64) - 127))
    return v * np.repeat(f, 32, axis=1)


def lay_out(codes, scale_bytes):
    """The stored arrays: codes [rows, Kp / 2] (element 2 j in the low half of
    byte j) and scales [Kp / 256, rows, 8], rows filled up with zeros to Kp."""
    rows, cols = codes.shape
    kp = -(-cols // 256) * 256
    c = np.zeros((rows, kp), np.uint8)
    c[:, :cols] = codes
    s = np.zeros((rows, kp // 32), np.uint8)
    s[:, : cols // 32] = scale_bytes
    return c[:, 0::2] | (c[:, 1::2] << 4), np.ascontiguousarray(s.reshape(rows, kp // 256, 8).transpose(1, 0, 2))


def quantized(x):
    """The values x stands for after rounding to MX4."""
    return values(*quantize(x))
