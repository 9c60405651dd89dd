"""Oracle of the operators between 4-bit linear layers, on the host: dropout's
random bits, the root-mean-square norm and its gradients in float64, and MXFP8
from its definition.

MXFP8: a block of 32 elements has one E8M0 byte b = floor(log2 max|x|) - 8 + 127,
at least 0, and E4M3FN codes, the nearest of x / 2^(b - 127) found by comparing
distances, ties to the even code, magnitudes beyond 448 becoming 448.  A block
with a NaN or an infinity is b = 255 with codes 0 and stands for NaN.  Storage:
codes [panels][rows][256], scales [panels][rows][8].
"""
import numpy as np

PANEL, BLOCK = 256, 32


# ---------------------------------------------------------------- dropout --

def philox(counter, key, rounds=10):
    """Philox4x32 of uint64 arrays that hold 32-bit words: counter (4 arrays or
    numbers), key (2 numbers)."""
    low = np.uint64(0xFFFFFFFF)
    c = [np.atleast_1d(np.asarray(v, np.uint64)) for v in counter]
    k = [int(v) for v in key]
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def drop_cut(p):
    return int(np.floor(p * 65536.0 + 0.5))


def drop_bits(rows, cols, seed, offset):
    """The 16 bits of every element."""
    out = np.zeros((rows, cols), np.uint32)
    seed, offset = int(seed) & (2 ** 64 - 1), int(offset) & (2 ** 64 - 1)
    for t in range(rows):
        c = np.arange(cols)
        w = philox((c // 8, t, offset & 0xFFFFFFFF, offset >> 32), (seed & 0xFFFFFFFF, seed >> 32))
        w = np.stack([np.broadcast_to(v, c.shape) for v in w])
        out[t] = (w[c // 2 % 4, c] >> (16 * (c % 2)).astype(np.uint64)) & np.uint64(0xFFFF)
    return out


def drop_factors(rows, cols, p, seed, offset):
    """What dropout multiplies every element by, in float64 (0 or the FP32 factor)."""
    cut = drop_cut(p)
    return np.where(drop_bits(rows, cols, seed, offset) >= cut, np.float64(np.float32(65536.0 / (65536.0 - cut))), 0.0)


# ------------------------------------------------------------------- norm --

def rms(h, eps):
    """1 / sqrt(mean(h^2) + eps) of each row, float64."""
    h = np.asarray(h, np.float64)
    return 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)


def norm(h, w, eps):
    return np.asarray(h, np.float64) * rms(h, eps)[:, None] * np.asarray(w, np.float64)


def norm_backward(dy, h, w, eps):
    """Gradients of norm(h, w, eps) for dy: (of h, of w)."""
    dy, h, w = (np.asarray(v, np.float64) for v in (dy, h, w))
    r = rms(h, eps)[:, None]
    u = h * r
    g = dy * w
    return r * (g - u * np.mean(g * u, axis=1, keepdims=True)), np.sum(dy * u, axis=0)


# ------------------------------------------------------------------ MXFP8 --

def e4m3_values():
    """The values of codes 0 .. 126, ascending."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e > 0, (1 + m / 8) * np.exp2(e.astype(np.float64) - 7), m / 8 * 2.0 ** -6)


def nearest_e4m3(a):
    """Code of the value nearest to a >= 0, ties to the even code."""
    v = e4m3_values()
    a = np.minimum(np.asarray(a, np.float64), v[-1])
    hi = np.clip(np.searchsorted(v, a), 1, 126)
    lo = hi - 1
    down, up = a - v[lo], v[hi] - a
    return np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi).astype(np.uint8)


def mx8_quantize(x):
    """(codes, scales) of x [rows][cols] blocked along its rows."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    p = -(-cols // PANEL)
    v = np.zeros((rows, p * PANEL))
    v[:, :cols] = x
    v = v.reshape(rows, p * 8, BLOCK)
    top = np.max(np.abs(v), axis=-1)
    byte = np.zeros(top.shape, np.int64)
    fine = np.isfinite(top)
    pos = fine & (top > 0)
    byte[pos] = np.maximum(np.floor(np.log2(top[pos])).astype(np.int64) - 8 + 127, 0)
    byte[~fine] = 255
    unit = np.exp2(np.where(fine, byte, 127).astype(np.float64) - 127)[..., None]
    safe = np.where(fine[..., None], v, 0.0)
    code = nearest_e4m3(np.abs(safe) / unit) | (np.signbit(safe).astype(np.uint8) << 7)
    return (np.ascontiguousarray(code.reshape(rows, p, PANEL).transpose(1, 0, 2)),
            np.ascontiguousarray(byte.astype(np.uint8).reshape(rows, p, 8).transpose(1, 0, 2)))


def mx8_dequantize(codes, scales, cols):
    p, rows, _ = codes.shape
    v = np.append(e4m3_values(), np.nan)[codes & 127] * np.where(codes & 128, -1.0, 1.0)
    unit = np.exp2(scales.astype(np.float64) - 127)
    unit[scales == 255] = np.nan
    v = v.reshape(p, rows, 8, BLOCK) * unit[..., None]
    return v.reshape(p, rows, PANEL).transpose(1, 0, 2).reshape(rows, -1)[:, :cols]
