"""FP8 matrices with block scales: quantization step by step, and products in float64.

Written from the definitions: E4M3 has four exponent bits (bias 7) and three of mantissa, its
largest value 448, its smallest 2^-9, and one NaN per sign (0x7F, 0xFF).
"""
import numpy as np

TOP = np.float32(448.0)
LEAST = np.float32(2.0 ** -100)


def values(codes):
    """E4M3 bytes -> float64."""
    b = codes.astype(np.int64)
    e, m = (b >> 3) & 15, (b & 7).astype(np.float64)
    v = np.where(e == 0, m * 2.0 ** -9, np.exp2(e - 7.0) * (1.0 + m / 8.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >> 7 == 1, -v, v)


def encode(x):
    """Nearest E4M3 byte of |x| <= 464, ties to even; NaN -> 0x7F. x: float64 holding the value to round."""
    x = np.asarray(x, np.float64)
    a = np.abs(np.where(np.isnan(x), 0.0, x))
    step = np.exp2(np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    v = np.rint(a / step) * step                       # np.rint: ties to even
    e = np.floor(np.log2(np.maximum(v, 2.0 ** -6)))
    m = v / np.exp2(e - 3)                             # 8 .. 15, or 0 .. 7 below 2^-6
    code = np.where(m >= 8, (e + 7) * 8 + (m - 8), m).astype(np.int64)
    code |= np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def blocks(n):
    return -(-n // 128)


def spread(scales, tall, shape):
    """Scales of blocks, one for every value of `shape`."""
    s = np.repeat(np.repeat(scales, 128, -1), tall, -2) if tall > 1 else np.repeat(scales, 128, -1)
    return s[..., :shape[-2], :shape[-1]]


def quantize(x, tall=1):
    """float32 [N][K] -> (codes, scales): every step one IEEE FP32 operation. tall: rows of a block."""
    x = np.asarray(x, np.float32)
    N, K = x.shape
    rows = -(-N // tall)
    y = np.zeros((rows * tall, blocks(K) * 128), np.float32)
    y[:N, :K] = x
    top = np.abs(y).reshape(rows, tall, blocks(K), 128).max((1, 3))
    s = np.maximum(top, LEAST) / TOP
    s = np.where(np.isfinite(top), s, np.float32(np.nan)).astype(np.float32)
    with np.errstate(invalid="ignore"):
        q = x / spread(s, tall, x.shape)
    q = np.where(np.isnan(q), np.nan, q.astype(np.float64))
    return encode(q), s


def silu_mul(x):
    """[M][2K], a gate beside a factor -> silu(gate) * factor in float64."""
    g, u = np.split(np.asarray(x, np.float64), 2, -1)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def product(a, a_scales, w, w_scales):
    """(A W^T in float64, the same of absolute values)."""
    x = values(a) * spread(a_scales.astype(np.float64), 1, a.shape)
    y = values(w) * spread(w_scales.astype(np.float64), 128, w.shape)
    return x @ y.T, np.abs(x) @ np.abs(y).T


def grouped(a, a_scales, w, w_scales, offsets, rows, out):
    """Products by expert into a copy of out (float64): (out, sums of absolute values, which rows were written)."""
    out = np.array(out, np.float64)
    size = np.zeros_like(out)
    hit = np.zeros(out.shape[0], bool)
    for e in range(len(offsets) - 1):
        for p in range(offsets[e], offsets[e + 1]):
            at = p if rows is None else rows[p]
            if 0 <= at < a.shape[0]:
                out[p], size[p] = (v[0] for v in product(a[at:at + 1], a_scales[at:at + 1], w[e], w_scales[e]))
                hit[p] = True
    return out, size, hit
