"""Plain numpy implementation of the microscaled 4-bit format (include/gq.h),
in 64 bits: the reference of its tests."""
import numpy as np

VALUES = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
# the ends of the values that round to each magnitude; True: the end itself
# rounds up (to the neighbour whose code is even)
ENDS = ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True),
        (5.0, False))


def blocks(cols):
    return -(-cols // 32)


def quantize(x, in_mul=1.0):
    """(scales [rows, nb], codes [rows, nb, 16]) of a float matrix."""
    with np.errstate(invalid="ignore", over="ignore"):
        g = np.asarray(x, np.float32) * np.float32(in_mul)
    rows, cols = g.shape
    nb = blocks(cols)
    p = np.zeros((rows, nb * 32), np.float64)
    p[:, :cols] = g
    p = p.reshape(rows, nb, 32)
    m = np.abs(p).max(2)                       # NaN where the block holds one
    bad = ~np.isfinite(m)
    frac, e = np.frexp(np.where(bad | (m == 0), 1.0, m))   # m = frac * 2^e, frac in [0.5, 1)
    s = np.maximum(0, e - 1 - 2 + 127)
    s[m == 0] = 0
    y = np.where(bad[..., None], 0.0, p) * np.exp2(127.0 - s)[..., None]
    a = np.abs(y)
    code = np.zeros(a.shape, np.uint8)
    for end, up in ENDS:
        code += (a >= end) if up else (a > end)
    code |= np.signbit(y).astype(np.uint8) << 3
    code[bad] = 0
    s = np.where(bad, 255, s).astype(np.uint8)
    return s, (code[..., 0::2] | code[..., 1::2] << 4)


def decode(s, q, cols):
    """Values [rows, cols] in 64 bits (NaN where the scale is 255)."""
    c = np.stack([q & 15, q >> 4], -1).reshape(q.shape[0], q.shape[1], 32)
    two = np.exp2(s.astype(np.float64) - 127)
    two[s == 255] = np.nan
    return (VALUES[c] * two[..., None]).reshape(q.shape[0], -1)[:, :cols]


def reduce(ss, qs, cols):
    """The rank-order sum, every sum rounded to binary32 (the values are
    exact in binary64, and so is a binary32 sum of two of them up to the one
    rounding)."""
    r = np.zeros((qs[0].shape[0], cols), np.float32)
    with np.errstate(invalid="ignore"):
        for s, q in zip(ss, qs):
            r = (r.astype(np.float64) + decode(s, q, cols)).astype(np.float32)
    return r
