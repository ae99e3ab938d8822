"""MXFP4 in numpy, 64 bits: written from the format's definition (blocks of 32,
scale 2^(floor(log2 max) - 2), e2m1 codes to nearest with ties to the even code)."""
import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
MID = (GRID[1:] + GRID[:-1]) / 2


def exponents(x):
    """Scale exponents of the blocks of 32 (256 stands for NaN)."""
    b = np.abs(np.asarray(x, np.float64)).reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    with np.errstate(invalid="ignore"):
        top = b.max(-1)
    bad = ~np.isfinite(b).all(-1)
    safe = np.where(bad | (top == 0), 1.0, top)
    e = np.maximum(np.frexp(safe)[1] - 1 - 2, -127)
    return np.where(bad, 256, np.where(top == 0, -127, e))


def round_e2m1(v):
    """Signed values to the nearest of the grid, ties to the even code, at most 6."""
    a = np.abs(v)
    down = np.searchsorted(MID, a, side="left")
    up = np.searchsorted(MID, a, side="right")
    code = np.where(down % 2 == 0, down, up)
    return np.copysign(GRID[code], v)


def with_exponents(x, e):
    """The values of x's codes under given block exponents."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    s = np.ldexp(1.0, np.where(e == 256, 0, e))[..., None]
    q = np.where((e == 256)[..., None], np.nan, round_e2m1(np.nan_to_num(b) / s) * s)
    return q.reshape(x.shape)


def quantize(x):
    """(values, scale bytes)."""
    e = exponents(x)
    return with_exponents(x, e), np.where(e == 256, 255, e + 127).astype(np.uint8)


def values(codes, scale):
    """The values that packed codes and scale bytes stand for."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    v = GRID[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def pack(vals, scale):
    """Packed codes of values that lie on the grid under the scale bytes."""
    s = np.repeat(np.ldexp(1.0, scale.astype(np.int64) - 127), 32, axis=-1)
    v = np.nan_to_num(np.asarray(vals, np.float64) / s)
    code = np.searchsorted(GRID, np.abs(v)).astype(np.uint8) | (np.signbit(v).astype(np.uint8) << 3)
    code = code.reshape(*code.shape[:-1], -1, 2)
    return (code[..., 0] | code[..., 1] << 4).astype(np.uint8)
