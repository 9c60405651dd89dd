"""MXFP4 oracle: the format from its definition, in float64 on the host.

A block of 32 elements has one E8M0 byte b, its elements E2M1 codes; the value
is x_E2M1 * 2^(b - 127).  The byte is floor(log2 max|x|) - 2 + 127, at least 0;
the codes are the nearest E2M1 magnitudes of |x| / 2^(b - 127), ties to the
even code, found here by comparing the distances to all eight.  A block with a
NaN or an infinity is b = 255 with codes 0 and stands for NaN.

Storage: panels of 256 elements along the blocked axis, codes
[panels][rows][128] (element 2i in the low nibble), scales [panels][rows][8];
elements behind a row's end are zeros.
"""
import numpy as np

PANEL, BLOCK = 256, 32
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def panels(n):
    return -(-n // PANEL)


def scale_byte(block_max):
    """E8M0 byte of a block from its largest magnitude (float64 scalar or array)."""
    m = np.atleast_1d(np.asarray(block_max, np.float64))
    byte = np.zeros(m.shape, np.int64)
    pos = (m > 0) & np.isfinite(m)
    byte[pos] = np.maximum(np.floor(np.log2(m[pos])).astype(np.int64) - 2 + 127, 0)
    byte[~np.isfinite(m)] = 255
    return byte


def nearest_code(a):
    """Nearest E2M1 magnitude code of a >= 0, ties to the even code (a above 6: 7)."""
    a = np.asarray(a, np.float64)
    out = np.zeros(a.shape, np.uint8)
    best = np.full(a.shape, np.inf)
    for c in (0, 2, 4, 6, 1, 3, 5, 7):        # even codes first: they keep a tie
        d = np.abs(a - E2M1[c])
        out[d < best] = c
        best = np.minimum(best, d)
    return out


def quantize(x):
    """(codes, scales) of x [rows][cols] blocked along its rows."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    p = panels(cols)
    v = np.zeros((rows, p * PANEL))
    v[:, :cols] = x
    v = v.reshape(rows, p * 8, BLOCK)
    with np.errstate(invalid="ignore"):
        top = np.max(np.abs(v), axis=-1)
    byte = scale_byte(top)
    bad = byte == 255
    unit = np.exp2(np.where(bad, 127, byte).astype(np.float64) - 127)[..., None]
    safe = np.where(bad[..., None], 0.0, v)
    code = nearest_code(np.abs(safe) / unit) | (np.signbit(safe).astype(np.uint8) << 3)
    code = code.reshape(rows, p, 128, 2)
    packed = (code[..., 0] | (code[..., 1] << 4)).astype(np.uint8)
    return (np.ascontiguousarray(packed.transpose(1, 0, 2)),
            np.ascontiguousarray(byte.astype(np.uint8).reshape(rows, p, 8).transpose(1, 0, 2)))


def dequantize(codes, scales, cols):
    """The float64 values [rows][cols] of an operand blocked along its rows."""
    p, rows, _ = codes.shape
    nib = np.stack((codes & 15, codes >> 4), -1).reshape(p, rows, 8, BLOCK)
    val = E2M1[nib & 7] * np.where(nib & 8, -1.0, 1.0)
    unit = np.exp2(scales.astype(np.float64) - 127)
    unit[scales == 255] = np.nan
    return (val * unit[..., None]).reshape(p, rows, PANEL).transpose(1, 0, 2).reshape(rows, -1)[:, :cols]


def held(x):
    """What x becomes when it is held in MXFP4 along its rows."""
    return dequantize(*quantize(x), np.asarray(x).shape[1])
