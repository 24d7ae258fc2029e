"""Sums of the block-scaled product whose large terms cancel, against float64.

Every group of eight neighbouring products of a row holds 64^2 and -64^2; the others lie between 0.25
and 0.4 and have one sign, so that their sum is the result.  With S = sum |A| |B|, u = 2^-24, scales and
all:
* a sum in fp32 of exact products, in any order, is within (K + K / 128 + 20) u S of the result: an
  addition for each product, the scales' product and the FMA of each run, the joins of split sums;
  S is some 5000 times the result, so the bound is a small share of it up to K = 2000;
* the result's rounding is half a step, 2^-8 (bf16) or u (fp32) of it.
A sum that drops what lies 13 bits below a group's largest product (2^12 / 2^13 = 0.5) loses every one of
the other terms, and the result with them.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mixture_experts_layer_31_amd as moe
from oracle import fp8_oracle as q8

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32, E4M3 = moe.MOE_TYPE_BF16, moe.MOE_TYPE_F32, moe.MOE_TYPE_E4M3
TILE, BLOCK = moe.MOE_SCALE_TILE, moe.MOE_SCALE_BLOCK
DT = {BF: torch.bfloat16, F32: torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    moe.lib()


def _operands(rng, M, N, K):
    """Values of A [M, K] and B [N, K], all of them e4m3's; every run of A has the amax 448, where B is 0."""
    small = np.array([0.5, 0.5625, 0.625])
    a, b = rng.choice(small, (M, K)), rng.choice(small, (N, K))
    for g in range(0, K - 7, 8):
        i, j, top = rng.choice(8, 3, replace=False)
        a[:, g + i] = a[:, g + j] = b[:, g + i] = 64
        b[:, g + j] = -64
        if g % 128 == 0:
            a[:, g + top], b[:, g + top] = 448, 0
    return a, b


def _scales(rng, *shape):
    return (1 + rng.integers(0, 4, shape) / 4).astype(np.float32)  # the scales' products are exact


def _spread(s, n, axis):
    return np.repeat(s.astype(np.float64), 128, axis=axis).take(range(n), axis=axis)


# one launch, 64 x 64 tiles with one group and two, 96, 128 and 256 rows a tile, whole and partial last
# runs, and a few rows past a multiple of 256
@pytest.mark.parametrize("M,N,K", [(1, 40, 128), (20, 33, 1000), (65, 67, 2000), (2000, 900, 300), (700, 256, 1040),
                                   (300, 700, 2000), (1500, 1900, 300), (2040, 2000, 520), (2048, 2048, 2000),
                                   (2900, 2890, 256), (2890, 2900, 300), (8195, 2048, 140)])
@pytest.mark.parametrize("a_type", [E4M3, BF, F32])
@pytest.mark.parametrize("b_scale", [TILE, BLOCK])
def test_small_terms_beside_outliers_that_cancel(M, N, K, a_type, b_scale):
    rng = np.random.default_rng(M + N + K)
    av, bv = _operands(rng, M, N, K)
    kb, ld = (K + 127) // 128, (K + 15) // 16 * 16
    quant = a_type != E4M3
    sa = np.ones((kb, M), np.float32) if quant else _scales(rng, kb, M)  # amax 448 in every run: a scale of 1
    sb = _scales(rng, kb, N) if b_scale == TILE else _scales(rng, (N + 127) // 128, kb)
    pad = lambda c: np.pad(c, ((0, 0), (0, ld - K)))  # noqa: E731
    b = torch.from_numpy(pad(q8.e4m3_encode(bv))).cuda()
    if quant:
        a, at = torch.from_numpy(av.astype(np.float32)).to(DT[a_type]).cuda(), None
    else:
        a, at = torch.from_numpy(pad(q8.e4m3_encode(av))).cuda(), torch.from_numpy(sa).cuda()
    va = av * _spread(sa.T, K, 1)
    vb = bv * (_spread(sb.T, K, 1) if b_scale == TILE else _spread(_spread(sb, N, 0), K, 1))
    ref, S = va @ vb.T, np.abs(va) @ np.abs(vb).T
    for ct in (BF, F32):
        print(f"[case] outliers {M}x{N}x{K} a={a_type} b_scale={b_scale} c={ct}", flush=True)
        c = torch.full((M, N), np.nan, dtype=DT[ct], device="cuda")
        d = moe.make_block_mm_desc(M, N, K, a_type=a_type, b_scale=b_scale, c_type=ct, ldb=ld)
        scratch = torch.full((max(1, moe.moe_block_mm_scratch_bytes(d)),), 0xA5, dtype=torch.uint8, device="cuda")
        assert moe.moe_block_mm(d, a, at, b, torch.from_numpy(sb).cuda(), c, scratch) == moe.MOE_OK
        torch.cuda.synchronize()
        bound = (K + K / 128 + 20) * U * S + (2.0 ** -8 if ct == BF else U) * np.abs(ref)
        err = np.abs(c.cpu().double().numpy() - ref)
        assert np.all(err <= bound), float((err / bound).max())
