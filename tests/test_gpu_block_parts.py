"""Contractions in parts with every tile size, whose sums a second launch joins, and added results at size."""
from __future__ import annotations

import pytest
import torch

import mixture_experts_layer_31_amd as moe
from tests import test_gpu_block as tb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    moe.lib()


# 64 x 64 tiles with one group of waves and with two, 96 x 128 and 128 x 128 (fp32), in 4 to 32 parts
@pytest.mark.parametrize("M,N,K", [(3000, 10, 5100), (8, 535, 12600), (70, 2800, 7200), (3000, 66, 15000), (834, 66, 44155)])
@pytest.mark.parametrize("b_scale", [tb.TILE, tb.BLOCK])
def test_parts(M, N, K, b_scale):
    for ct in (tb.BF, tb.F32):
        assert moe.moe_block_mm_scratch_bytes(moe.make_block_mm_desc(M, N, K, b_scale=b_scale, c_type=ct)) >= 4 * 4 * M * N
        tb._check_mm(M, N, K, b_scale, ct, seed=K, ldc=N + 3, off=1, add=ct == tb.F32)


@pytest.mark.parametrize("M,N,K", [(2040, 2000, 520), (2048, 2048, 8192), (8200, 2048, 300)])
@pytest.mark.parametrize("b_scale", [tb.TILE, tb.BLOCK])
def test_tiles_of_128_rows_and_more(M, N, K, b_scale):
    tb._check_mm(M, N, K, b_scale, tb.BF, seed=7, ldc=N + 1, off=1)
    tb._check_mm(M, N, K, b_scale, tb.F32, seed=8, add=True)
