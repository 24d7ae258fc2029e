"""One AdamW step over one tensor in float64, and its states' e4m3 form.  TEST INFRASTRUCTURE ONLY."""
from __future__ import annotations

import numpy as np

from oracle import fp8_oracle as q8


def step(p, g, m, v, lr, t, beta1, beta2, eps, decay, norm=None, max_norm=0.0):
    """(p, m, v) after the step, of arrays in float64."""
    p, g, m, v = (np.asarray(x, np.float64) for x in (p, g, m, v))
    if t < 1 or (norm is not None and not np.isfinite(norm)):
        return p, m, v
    if norm is not None and norm > max_norm:
        g = g * (max_norm / norm)
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    p = p * (1 - lr * decay) - lr * (m / (1 - beta1 ** t)) / (np.sqrt(v / (1 - beta2 ** t)) + eps)
    return p, m, v


def moments32(g, m, v, beta1, beta2, norm=None, max_norm=0.0):
    """(m, v) in float32 as they are defined: each quotient, product and sum rounded."""
    f = np.float32
    g, m, v = (np.asarray(x, f) for x in (g, m, v))
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        if norm is not None and f(norm) > f(max_norm):
            g = g * (f(max_norm) / f(norm))
        return (f(beta1) * m + f(1 - beta1) * g, f(beta2) * v + f(1 - beta2) * (g * g))


def encode(x, least=False):
    """(codes uint8, scales fp32) of x, fp32 values, in runs of 128; least: what is positive has a code of 1 at least.  A scale
    amax / 448 that rounds to 0 is 1, and the codes are zeros; a NaN, which amax passes over, is 0x7F."""
    x = np.asarray(x, np.float32)
    n = x.size
    t = np.pad(x, (0, -n % 128)).reshape(-1, 128)
    s = (np.fmax.reduce(np.abs(t), axis=1, initial=0) / np.float32(448)).astype(np.float32)
    s = np.where(s == 0, np.float32(1), s)
    with np.errstate(invalid="ignore"):
        q = (t / s[:, None]).astype(np.float32)
    codes = np.where(np.isnan(q), 0x7F, q8.e4m3_encode(q))
    if least:
        codes = np.where((t > 0) & (codes == 0), 1, codes)
    return codes.astype(np.uint8).reshape(-1)[:n], s


def decode(codes, scales):
    """The values: code * scale in float32."""
    codes = np.asarray(codes, np.uint8)
    return q8.e4m3_decode(codes).astype(np.float32) * np.repeat(np.asarray(scales, np.float32), 128)[:codes.size]
