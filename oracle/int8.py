"""fp64 codecs of 8-bit integers: rows with one scale each, and OCP MXINT8
(one E8M0 scale per 32 consecutive elements, value = code * scale / 64)."""
from __future__ import annotations

import numpy as np

__all__ = ["quantize_int8", "quantize_mxint8", "decode_mxint8"]


def _nearest_even(halves):
    """The whole number nearest to halves / 2 for halves >= 0; where halves is an odd whole number, the even one."""
    n = np.floor((halves + 1.0) / 2.0)
    return n - ((halves == 2.0 * n - 1.0) & (n % 2 == 1))


def quantize_int8(x):
    """x [rows, K] -> (codes int8, scales fp32 [rows]): scale = fp32(amax / 127),
    at least 2^-126, at most the largest fp32 number whose 127-fold is finite, 1
    for zeros; code = 127 x / amax (2^126 x at the least
    scale). Of inputs of at most 24 bits, the fp64 quotient of an exact product
    falls on a tie exactly where the true one does. A row with an infinite or
    NaN element: scale NaN, codes 0."""
    x = np.asarray(x, dtype=np.float64)
    finite = np.isfinite(x).all(axis=1)
    v = np.where(finite[:, None], x, 0.0)
    amax = np.abs(v).max(axis=1)
    tiny = amax < 127.0 * 2.0 ** -126
    den = np.where(tiny, 127.0 * 2.0 ** -126, amax)
    code = np.sign(v) * _nearest_even(254.0 * np.abs(v) / den[:, None])
    most = np.float32(np.finfo(np.float32).max / 127.0)
    if float(most) * 127.0 > float(np.finfo(np.float32).max):
        most = np.nextafter(most, np.float32(0))
    scale = np.where(tiny, np.float32(2.0 ** -126), np.minimum((den / 127.0).astype(np.float32), most))
    scale = np.where(amax == 0, np.float32(1.0), scale)
    return code.astype(np.int8), np.where(finite, scale, np.float32(np.nan)).astype(np.float32)


def quantize_mxint8(x):
    """x [rows, K] -> (codes int8, E8M0 bytes [rows, K/32]): scale 2^floor(log2
    amax), at least 2^-120 (byte 7), 1 for zeros; code = 64 x / scale, at most 127
    in magnitude. A block with an infinite or NaN element: byte 255, codes 0."""
    x = np.asarray(x, dtype=np.float64)
    R, K = x.shape
    b = x.reshape(R, K // 32, 32)
    finite = np.isfinite(b).all(axis=2)
    v = np.where(finite[..., None], b, 0.0)
    amax = np.abs(v).max(axis=2)
    e = np.where(amax > 0, np.maximum(np.frexp(amax)[1] - 1, -120), 0)
    halves = np.abs(v) * np.exp2(7.0 - e)[..., None]
    code = np.sign(v) * np.minimum(_nearest_even(halves), 127.0)
    return code.reshape(R, K).astype(np.int8), np.where(finite, e + 127, 255).astype(np.uint8)


def decode_mxint8(codes, scales):
    codes, scales = np.asarray(codes), np.asarray(scales)
    step = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 133.0))
    return codes.astype(np.float64) * np.repeat(step, 32, axis=1)
