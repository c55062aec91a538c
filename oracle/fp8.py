"""CPU oracle of the e4m3 formats and the operators on them, in numpy: the
definitions in 64 bits, and the rounding rules in the IEEE fp32 steps that the
header states.  Shares no code with the HIP library.

Formats: e4m3 codes are bytes (sign, 4 exponent bits with bias 7, 3 mantissa
bits, no infinities, 0x7f and 0xff NaN); rows have a float32 scale for each
128 values, matrices one for each 128 x 128 block."""
from __future__ import annotations

import numpy as np

BLOCK = 128
SCALE_MIN = np.float32(2.0 ** -126)


def _decode_table() -> np.ndarray:
    t = np.empty(256, np.float64)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t[c] = (-1.0 if c & 128 else 1.0) * (np.nan if c & 127 == 127 else v)
    return t


DECODE = _decode_table()


def decode(codes) -> np.ndarray:
    return DECODE[np.asarray(codes, np.uint8)]


def encode(v) -> np.ndarray:
    """The nearest e4m3 code of finite |v| < 464, ties to the even mantissa."""
    v = np.asarray(v, np.float64)
    mag = DECODE[:127]                               # ascending: 0 .. 448
    at = np.clip(np.searchsorted(mag, np.abs(v)), 1, 126)
    below, above = mag[at - 1], mag[at]
    lo, hi = np.abs(v) - below, above - np.abs(v)
    code = np.where((hi < lo) | ((hi == lo) & (at % 2 == 0)), at, at - 1)
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def quantize(v):
    """fp32 rows -> (codes, scales) by the header's rule, step for step."""
    v = np.asarray(v, np.float32)
    T, C = v.shape
    p = np.zeros((T, blocks(C) * BLOCK), np.float32)
    p[:, :C] = v
    p = p.reshape(T, -1, BLOCK)
    a = np.maximum(np.abs(p).max(2), np.float32(448) * SCALE_MIN)
    q = p * (np.float32(448) / a)[..., None]
    return encode(q).reshape(T, -1)[:, :C], a / np.float32(448)


def rows(codes, scales) -> np.ndarray:
    """Values of e4m3 rows in 64 bits."""
    c = decode(codes)
    return c * np.repeat(np.asarray(scales, np.float64), BLOCK, 1)[:, :c.shape[1]]


def matrix(codes, scales) -> np.ndarray:
    """Values of an e4m3 matrix in 64 bits."""
    c = decode(codes)
    s = np.repeat(np.repeat(np.asarray(scales, np.float64), BLOCK, 0), BLOCK, 1)
    return c * s[:c.shape[0], :c.shape[1]]


def dense(x_codes, x_scales, w_codes, w_scales):
    """(y, the sum of its terms' magnitudes), both in 64 bits."""
    x, w = rows(x_codes, x_scales), matrix(w_codes, w_scales)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def silu_product(g, u) -> np.ndarray:
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def rmsnorm(x, weight, eps, residual=None):
    """(v, y): the fp32 sum v of x and residual, and its norm times weight in 64 bits."""
    v = np.asarray(x, np.float32)
    if residual is not None:
        v = v + np.asarray(residual, np.float32)
    d = v.astype(np.float64)
    return v, d / np.sqrt((d * d).mean(1, keepdims=True) + float(np.float32(eps))) * np.asarray(weight, np.float64)
