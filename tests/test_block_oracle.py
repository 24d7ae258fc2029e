"""Pins of the block-scaled oracle: the FP8 layer's quantisers on whole blocks, closed forms on partial ones."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import block_oracle as bk
from oracle import fp8_oracle as q8


def _x(seed, R, C):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal((R, C)) * np.exp2(rng.uniform(-9, 9, (R, 1)))).astype(np.float32)


def test_whole_runs_are_the_layers():
    x = _x(1, 5, 384)
    c, s = bk.quant_tiles(x)
    wc, ws = q8.quant_rows(x, 128, False)
    assert np.array_equal(c, wc) and np.array_equal(s, np.asarray(ws, np.float32).T)


@pytest.mark.parametrize("R,C", [(1, 1), (3, 130), (129, 100), (256, 257)])
def test_partial_blocks_against_torch(R, C):
    """Each run and block alone, with torch's division and e4m3 cast."""
    x = _x(R * 1000 + C, R, C)
    for quant, rows, scale_of in ((bk.quant_tiles, 1, lambda s, i, j: s[j, i]), (bk.quant_blocks, 128, lambda s, i, j: s[i, j])):
        codes, scales = quant(x)
        assert codes.shape == (R, C)
        for i in range(0, R, rows):
            for j in range(0, C, 128):
                part = torch.from_numpy(x[i:i + rows, j:j + 128])
                s = part.abs().max() / 448
                assert scale_of(scales, i // rows, j // 128) == s.item()
                want = (part / s).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
                assert np.array_equal(codes[i:i + rows, j:j + 128], want)


def test_zeros_and_tiny_values():
    c, s = bk.quant_tiles(np.zeros((2, 200), np.float32))
    assert not c.any() and (s == 1).all()
    x = np.full((1, 3), 2.0 ** -149, np.float32)  # amax / 448 rounds to 0: the scale is 1
    c, s = bk.quant_blocks(x)
    assert not c.any() and (s == 1).all()


def test_values_come_back():
    """A value is off by half a step of its code: 2^-4 relative, or 2^-10 of its scale below the normal codes."""
    x = _x(7, 150, 300)
    for quant, values, scale in ((bk.quant_tiles, bk.values_tiles, lambda s: np.repeat(s.T, 128, 1)[:, :300]),
                                 (bk.quant_blocks, bk.values_blocks,
                                  lambda s: np.repeat(np.repeat(s, 128, 0), 128, 1)[:150, :300])):
        c, s = quant(x)
        # and the fp32 scale's own rounding, 2^-24
        assert np.all(np.abs(values(c, s) - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * scale(s)) * (1 + 2 ** -20))
