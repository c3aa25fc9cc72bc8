"""The 8-bit cache's format in float64, the oracle of its operators.

TEST INFRASTRUCTURE ONLY (see the package docstring): nothing on the CUDA path imports this.

A row (the values of one position and key-value head) is e4m3 codes and one e8m0 byte,
value = code * 2^(byte - 127); NaN throughout where the byte is 255.
"""
from __future__ import annotations

import numpy as np

from oracle.numerics import E4M3_MAX, e4m3_to_f64, f32_to_e4m3_rne

#: The smallest exponent of a scale, and the byte of a row with an infinity or NaN.
MIN_EXPONENT = -100
NAN_SCALE = 255


def quantise(x):
    """Codes and bytes of the rows x [..., D] (float64): the smallest power of two, from 2^-100 on,
    for which no value exceeds 448 times it; 1 for a row of zeros."""
    x = np.asarray(x, dtype=np.float64)
    finite = np.isfinite(x).all(-1)
    top = np.abs(np.where(finite[..., None], x, 0.0)).max(-1)
    e = np.full(top.shape, MIN_EXPONENT)
    for n in range(MIN_EXPONENT, 130):      # one up while the row does not fit
        e = np.where(top > E4M3_MAX * np.ldexp(1.0, n), n + 1, e)
    e = np.where(top == 0, 0, e)
    codes = f32_to_e4m3_rne(np.where(finite[..., None], x, 0.0) / np.ldexp(1.0, e)[..., None])
    codes = np.where(finite[..., None], codes, 0).astype(np.uint8)
    return codes, np.where(finite, e + 127, NAN_SCALE).astype(np.uint8)


def values(codes, scales):
    """The values of rows; bytes below that of 2^-100 count as it."""
    s = np.asarray(scales).astype(np.int64)
    f = np.ldexp(1.0, np.maximum(s, MIN_EXPONENT + 127) - 127)
    return e4m3_to_f64(codes) * np.where(s == NAN_SCALE, np.nan, f)[..., None]
