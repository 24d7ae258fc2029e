"""Products that quantise A themselves, with either scale layout of B and either type of result.

Against the float64 product of the codes' values, which are the oracle's of A's values: fp32 sums of exact
products, (128 + K / 128 + 20) u S with S = sum |A| |B| and u = 2^-24, and the result's rounding, 2^-8 of it in bf16
and u in fp32.  Where the product of the codes that moe_block_quant gives takes the same kernel, its bits are
the same too; where it takes another one, the sums may have another order.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mixture_experts_layer_31_amd as moe
from oracle import block_oracle as bk
from tests import test_gpu_block as tb

pytestmark = pytest.mark.gpu
BF, F32, TILE, BLOCK = tb.BF, tb.F32, tb.TILE, tb.BLOCK
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    moe.lib()


# one launch for values and for codes; one launch for values alone; tiles of 64, 96, 128 and 256 rows, rows
# past a multiple of 256, and enough rows for two a thread in the quantiser
SAME = [(1, 64, 300), (2, 70, 1000), (50, 256, 520), (500, 300, 900), (1500, 1900, 300), (2040, 2000, 520),
        (2900, 2890, 300), (8200, 2048, 140), (16400, 260, 1030)]


@pytest.mark.parametrize("M,N,K", SAME + [(64, 6000, 512)])
@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("b_scale", [TILE, BLOCK])
def test_values(M, N, K, t, b_scale):
    x = tb._x(M + N, M, K, t, spread=1.0)
    va = bk.values_tiles(*bk.quant_tiles(x.float().numpy()))
    b, sb, vb, ldb = tb._codes(2, N, K, b_scale)
    ref, S = va @ vb.T, np.abs(va) @ np.abs(vb).T
    ld = K + 3  # rows at any element
    xd = tb._strided(x, ld, off=1, fill=np.nan)
    ldq = (K + 15) // 16 * 16
    q = torch.full((M, ldq), 0x7F, dtype=torch.uint8, device="cuda")
    s = torch.full(((K + 127) // 128, M), np.nan, device="cuda")
    assert moe.moe_block_quant(moe.make_block_quant_desc(M, K, t, ld_in=ld), xd, q, s) == moe.MOE_OK
    for ct in (BF, F32):
        print(f"[case] values {M}x{N}x{K} t={t} b_scale={b_scale} c={ct}", flush=True)
        out = []
        for a, sa, at, lda in ((xd, None, t, ld), (q, s, moe.MOE_TYPE_E4M3, ldq)):
            c = torch.full((M, N + 2), 77.0, dtype=tb.DT[ct], device="cuda")
            d = moe.make_block_mm_desc(M, N, K, a_type=at, b_scale=b_scale, c_type=ct, lda=lda, ldb=ldb, ldc=N + 2)
            scratch = torch.full((max(1, moe.moe_block_mm_scratch_bytes(d)),), 0xFF, dtype=torch.uint8, device="cuda")
            assert moe.moe_block_mm(d, a, sa, b, sb, c, scratch) == moe.MOE_OK
            torch.cuda.synchronize()
            assert (c[:, N:] == 77).all()
            out.append(c[:, :N])
        bound = (128 + K / 128 + 20) * U * S + (2.0 ** -8 if ct == BF else U) * np.abs(ref) + 2.0 ** -126
        for c in out:
            assert np.all(np.abs(c.cpu().double().numpy() - ref) <= bound)
        if (M, N, K) in SAME:
            assert torch.equal(*out)


@pytest.mark.parametrize("t", [BF, F32])
def test_rows_of_many_values(t):
    """Two rows a thread: from 8192 slabs of 16 rows and a run on."""
    tb._check_quant(tb._x(7, 16400, 1030, t), t, "many rows", cols=False, ld=1033, off=1)
