"""MXFP4 codec, the paged cache's byte order, and attention over cached values (float64 / integers).

E2M1: values 0, .5, 1, 1.5, 2, 3, 4, 6 for the codes 0..7, negative with bit 3 set. A block of 32
elements along head_dim shares a power of two 2^e, stored as the byte e + 127: RCEIL takes the
smallest e with amax <= 6 * 2^e, FLOOR e = floor(log2 amax) - 2, both clamped to [-127, 127], and
amax = 0 gives byte 0. The code is the nearest value to x * 2^-e, ties to the even code, magnitudes
above 6 saturating, sign kept.

Byte order of a row: element 32 b + 4 g + 2 j + n (b < 4, g < 8, j < 2) is the low (n = 0) or high
(n = 1) nibble of byte 8 g + 2 b + j.

Parity: the codec is pinned by nearest search over all codes and exponents, the byte order by a loop
over its definition, the attention by a pure-Python softmax (CPU tests).
"""
from __future__ import annotations

import math

import numpy as np

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def decode(codes):
    """Codes (nibbles) -> float64."""
    c = np.asarray(codes).astype(np.int64)
    return VALUES[c & 7] * np.where(c & 8, -1.0, 1.0)


def encode(x):
    """float64 -> codes: nearest value, ties to the even code, saturating."""
    x = np.asarray(x, dtype=np.float64)
    mids = (VALUES[1:] + VALUES[:-1]) / 2
    a = np.abs(x)
    up = np.searchsorted(mids, a, side="right")      # a tie goes up ...
    tie = (up > 0) & (a == mids[np.maximum(up, 1) - 1])
    code = np.where(tie & (up % 2 == 1), up - 1, up)  # ... unless the lower code is the even one
    return (code + np.where(np.signbit(x), 8, 0)).astype(np.uint8)


def scale_exponent(amax, mode="rceil"):
    amax = np.asarray(amax, dtype=np.float64)
    m, x = np.frexp(np.where(amax > 0, amax, 1.0))    # amax = m 2^x, m in [.5, 1)
    e = x - 1 - 2
    if mode == "rceil":
        e = e + (2 * m > 1.5)
    return np.where(amax > 0, np.clip(e, -127, 127), -127).astype(np.int64)


def quantize_rows(x, mode="rceil"):
    """(..., 128) -> (codes (..., 128) uint8, exponents (..., 4))."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(x.shape[:-1] + (4, 32))
    e = scale_exponent(np.abs(b).max(axis=-1), mode)
    return encode(b * np.ldexp(1.0, -e)[..., None]).reshape(x.shape), e


def pack_rows(codes):
    """Codes (..., 128) -> bytes (..., 64) in the cache's order."""
    c = np.asarray(codes, dtype=np.uint8).reshape(codes.shape[:-1] + (4, 8, 2, 2))
    c = np.swapaxes(c, -4, -3)                          # (g, b, j, n)
    return (c[..., 0] | (c[..., 1] << 4)).reshape(codes.shape[:-1] + (64,))


def unpack_rows(data):
    """Bytes (..., 64) -> codes (..., 128)."""
    d = np.asarray(data, dtype=np.uint8).reshape(data.shape[:-1] + (8, 4, 2))
    c = np.stack([d & 15, d >> 4], axis=-1)
    return np.swapaxes(c, -4, -3).reshape(data.shape[:-1] + (128,))


def cached_rows(payload, scales, table_row, n, head, page_size):
    """The float64 values of the first n cached tokens of one head: payload (pages, H, page, 64)."""
    at = np.arange(n)
    page, row = np.asarray(table_row)[at // page_size], at % page_size
    v = decode(unpack_rows(payload[page, head, row]))
    e = scales[page, head, row].astype(np.int64) - 127
    return v * np.repeat(np.ldexp(1.0, e), 32, axis=-1)


def attend(q, k, v):
    """One query row q (128,) over keys k, v (n, 128): (O, LSE, mean |v| weight, largest sum |q k|)."""
    if not len(k):
        return np.zeros(128), -math.inf, np.zeros(128), 0.0
    s = k @ q / math.sqrt(128.0)
    m = s.max()
    p = np.exp(s - m)
    l = p.sum()
    return p @ v / l, m + math.log(l), p @ np.abs(v) / l, float((np.abs(k) @ np.abs(q)).max()) / math.sqrt(128.0)
