"""Block-scaled e4m3 matrices with partial last blocks, and their product, in float64.  TEST INFRASTRUCTURE ONLY.

The encodings and the scale rule are fp8_oracle's (fp32 scale amax / 448, 1 where that is 0; code
e4m3(x / scale)); here the last run or block of a row may be partial, and a scale that rounds to 0
is 1 too.
"""
from __future__ import annotations

import numpy as np

from oracle import fp8_oracle as q8


def _blocks(x, rows, cols):
    """(codes [R, C], scales [ceil(R/rows), ceil(C/cols)]) of x in blocks of rows x cols."""
    x = np.asarray(x, np.float32)
    R, C = x.shape
    rb, cb = -(-R // rows), -(-C // cols)
    t = np.zeros((rb * rows, cb * cols), np.float32)
    t[:R, :C] = x
    t = t.reshape(rb, rows, cb, cols)
    s = (np.abs(t).max(axis=(1, 3)).astype(np.float32) / np.float32(448)).astype(np.float32)
    s = np.where(s == 0, np.float32(1), s)
    codes = q8.quant_block(t, s[:, None, :, None]).reshape(rb * rows, cb * cols)[:R, :C]
    return codes, s


def quant_tiles(x):
    """(codes [R, C], scales [ceil(C/128), R])"""
    c, s = _blocks(x, 1, 128)
    return c, s.T.copy()


def quant_blocks(x):
    """(codes [R, C], scales [ceil(R/128), ceil(C/128)])"""
    return _blocks(x, 128, 128)


def values_tiles(codes, scales):
    return q8.e4m3_decode(codes) * np.repeat(scales.T.astype(np.float64), 128, axis=1)[:, :codes.shape[1]]


def values_blocks(codes, scales):
    s = np.repeat(np.repeat(scales.astype(np.float64), 128, axis=0), 128, axis=1)
    return q8.e4m3_decode(codes) * s[:codes.shape[0], :codes.shape[1]]
