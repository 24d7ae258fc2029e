"""Pins of AdamW's e4m3 states (oracle/adamw_oracle.py) where their scales leave fp32's normal numbers."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import adamw_oracle as ao

ULP = np.float32(2.0 ** -149)  # fp32's smallest number


@pytest.mark.parametrize("amax", [1, 2, 100, 223, 224, 225, 447, 448, 449, 671, 672, 673, 700, 5000])
def test_runs_of_subnormal_values(amax):
    """A scale that rounds to 0 (amax / 448 of at most half the smallest number) is 1 and the codes are zeros; no
    quotient is 0 / 0, and every value decodes to a number."""
    k = np.random.default_rng(amax).integers(-amax, amax + 1, 128)
    k[:3] = 0, amax, -amax
    x = k.astype(np.float32) * ULP
    codes, s = ao.encode(x)
    assert s[0] == (1 if amax <= 224 else max(1, round(amax / 448)) * ULP)
    assert not np.any((codes & 0x7F) == 0x7F)
    got = ao.decode(codes, s)
    assert got[0] == 0 and np.isfinite(got).all()
    if amax <= 224:
        assert not (codes & 0x7F).any() and np.array_equal(codes >= 0x80, k < 0)
    else:  # half a step of e4m3, or what passes 448 of the rounded scale, and half the smallest number for the product
        assert np.all(np.abs(got.astype(np.float64) - x) <= np.maximum(np.abs(x) / 16, np.abs(x) - 448 * s[0].astype(np.float64)) + ULP
                      + s[0].astype(np.float64) * 2.0 ** -10)
    # the second moment's root cannot be this small: a run of the smallest squares
    codes, s = ao.encode(np.sqrt(np.abs(x)), least=True)
    assert np.array_equal(codes > 0, k != 0) and s[0] > 0


def test_a_thousand_steps_without_a_gradient():
    """An expert that gets no tokens: its first moment shrinks to nothing and stays a number."""
    rng = np.random.default_rng(1)
    m = (rng.standard_normal((64, 128)) * 3e-4).astype(np.float32)
    m[:, 5] = 0
    codes, s = ao.encode(m.reshape(-1))
    zero = np.zeros(m.size, np.float32)
    top = np.inf
    for _ in range(1000):
        m32, _ = ao.moments32(zero, ao.decode(codes, s), zero, 0.9, 0.95)
        assert np.isfinite(m32).all() and np.abs(m32).max() <= top
        top = np.abs(m32).max()
        codes, s = ao.encode(m32)
    assert top < 1e-40 and not np.any((codes & 0x7F) == 0x7F)


def test_what_is_no_number_has_a_code_of_its_own():
    x = np.zeros(200, np.float32)
    x[3], x[4], x[130], x[131] = np.nan, 2.0, np.inf, 1.0
    codes, s = ao.encode(x)
    assert codes[3] == 0x7F and codes[4] == 0x7E and s[0] == np.float32(2) / np.float32(448)
    assert s[1] == np.inf and codes[130] == 0x7F and codes[131] == 0 and np.isnan(ao.decode(codes, s)[128:]).all()
