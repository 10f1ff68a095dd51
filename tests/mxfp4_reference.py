"""4-bit codes with an exponent byte for each 32 values, on the CPU in float64 from the definition."""
import numpy as np

VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def decode(codes, scales):
    """float64 values [..., n] of codes [..., n / 2] and scales [..., n / 32]."""
    both = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1).astype(np.int64)
    v = np.where(both >= 8, -1.0, 1.0) * VALUES[both & 7]
    with np.errstate(invalid="ignore"):
        scale = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
        return (v.reshape(*scales.shape, 32) * scale[..., None]).reshape(v.shape)


def encode(values):
    """(codes, scales) of float32 values [..., n]: the nearest of the sixteen by distance, ties to the even code."""
    x = np.ascontiguousarray(values, np.float64).reshape(-1, 32)
    finite = np.isfinite(x).all(1)
    x = np.where(finite[:, None], x, 0.0)
    top = np.abs(x).max(1)
    byte = np.zeros(len(x), np.int64)
    while True:                         # the least byte with top <= 6 * 2^(byte - 127)
        more = top > 6 * np.ldexp(1.0, byte - 127)
        if not more.any():
            break
        byte += more
    r = np.abs(x) / np.ldexp(1.0, byte - 127)[:, None]
    code = np.zeros(x.shape, np.int64)
    for c in range(1, 8):               # over the middle, or on it with an even code above
        middle = (VALUES[c - 1] + VALUES[c]) / 2
        code = np.where((r > middle) | ((r == middle) & (c % 2 == 0)), c, code)
    code = code + 8 * np.signbit(x)
    code[~finite] = 0
    byte[~finite] = 255
    code = code.reshape(*values.shape[:-1], -1, 2).astype(np.uint8)
    return code[..., 0] | (code[..., 1] << 4), byte.astype(np.uint8).reshape(*values.shape[:-1], -1)
