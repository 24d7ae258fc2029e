"""Products whose scales are large, small or subnormal, against float64.

The result is sum over the runs of sA sB P; sA sB alone may be infinite, 0 or of few bits where the result is
an ordinary number.  With S = sum |A| |B| over an output's values and u = 2^-24: fp32 sums of exact products,
both scales and the sum over the runs are within (128 + K / 128 + 20) u S of it, and the result's rounding is
half a step (2^-8 of it in bf16, u in fp32).  Below fp32's normal numbers a rounding is up to 2^-149 instead:
one for each run, one for the result, which bf16 rounds by up to 2^-134.  Results past fp32's (bf16's) range
are infinite.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mixture_experts_layer_31_amd as moe
from oracle import fp8_oracle as q8

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = moe.MOE_TYPE_BF16, moe.MOE_TYPE_F32
TILE, BLOCK = moe.MOE_SCALE_TILE, moe.MOE_SCALE_BLOCK
DT = {BF: torch.bfloat16, F32: torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    moe.lib()


def _wide(s, n, axis):
    return np.repeat(s.astype(np.float64), 128, axis=axis).take(range(n), axis=axis)


def _check(c, va, vb, K, ct, name):
    ref, S = va @ vb.T, np.abs(va) @ np.abs(vb).T
    kb = (K + 127) // 128
    bound = (128 + K / 128 + 20) * U * S + (2.0 ** -8 if ct == BF else U) * np.abs(ref) + (kb + 1) * 2.0 ** -149
    if ct == BF:
        bound += 2.0 ** -134
    got = c.cpu().double().numpy()
    # at (50, 50) and K = 9000 S is up to 2^102 448^2 9000 = 2^133: a result past the range is infinite, and one
    # whose S passes it may be
    assert np.isinf(got[np.abs(ref) >= 2.0 ** 129]).all(), name
    inside = S < 2.0 ** 127
    assert np.isfinite(got[inside]).all(), (name, int((~np.isfinite(got[inside])).sum()))
    err = np.abs(got - ref)[inside]
    assert np.all(err <= bound[inside]), (name, float((err / bound[inside]).max()))


# exponents of A's and B's scales, and the codes' sizes: large (normal), or 0 and 2^-9
EXPONENTS = [(-75, -72, "large"), (-90, -57, "large"), (-140, 100, "large"), (-149, 119, "large"), (119, -119, "large"),
             (50, 50, "large"), (63, 66, "small"), (119, 12, "small"), (20, 110, "small"), (-60, -55, "small"), (3, -2, "large")]


# one launch, 64 x 64 tiles with one group and two, parts, 96, 128 and 256 rows a tile
@pytest.mark.parametrize("M,N,K", [(1, 40, 300), (20, 33, 1000), (2000, 900, 300), (700, 256, 1040), (200, 129, 9000),
                                   (1500, 1900, 300), (2040, 2000, 520), (2890, 2900, 300), (8195, 2048, 140)])
@pytest.mark.parametrize("b_scale", [TILE, BLOCK])
def test_scales_of_any_size(M, N, K, b_scale):
    kb, ld = (K + 127) // 128, (K + 15) // 16 * 16
    rng = np.random.default_rng(M + N + K)
    big = M * N > 10 ** 6
    for ea, eb, size in EXPONENTS[::3] if big else EXPONENTS:
        mant = lambda e, *s: (2.0 ** e * (1 + rng.random(s))).astype(np.float32)  # noqa: E731
        sa = mant(ea, kb, M)
        sb = mant(eb, kb, N) if b_scale == TILE else mant(eb, (N + 127) // 128, kb)
        top = 0x7F if size == "large" else 0x02
        ca, cb = (rng.integers(0x60 if size == "large" else 0, top, (r, ld), dtype=np.uint8) for r in (M, N))
        for c in (ca, cb):
            c |= (rng.random(c.shape) < 0.2).astype(np.uint8) << 7
        va = q8.e4m3_decode(ca[:, :K]) * _wide(sa.T, K, 1)
        vb = q8.e4m3_decode(cb[:, :K]) * (_wide(sb.T, K, 1) if b_scale == TILE else _wide(_wide(sb, N, 0), K, 1))
        dev = [torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in (ca, sa, cb, sb)]
        for ct in (BF, F32):
            name = f"scales {M}x{N}x{K} 2^{ea} 2^{eb} {size} b_scale={b_scale} c={ct}"
            print("[case]", name, flush=True)
            c = torch.full((M, N), np.nan, dtype=DT[ct], device="cuda")
            d = moe.make_block_mm_desc(M, N, K, b_scale=b_scale, c_type=ct)
            scratch = torch.full((max(1, moe.moe_block_mm_scratch_bytes(d)),), 0xA5, dtype=torch.uint8, device="cuda")
            assert moe.moe_block_mm(d, *dev, c, scratch) == moe.MOE_OK
            torch.cuda.synchronize()
            _check(c, va, vb, K, ct, name)


@pytest.mark.parametrize("M,N,K", [(3, 40, 300), (2000, 900, 300), (700, 256, 520), (1500, 1900, 300), (2040, 2000, 520),
                                   (2890, 2900, 300)])
@pytest.mark.parametrize("b_scale", [TILE, BLOCK])
def test_runs_of_zeros_under_any_scales(M, N, K, b_scale):
    """A run whose sum is 0 adds 0, also where the scales' product is past the range; scales of 0 too."""
    kb, ld = (K + 127) // 128, (K + 15) // 16 * 16
    rng = np.random.default_rng(K)
    top = np.float32(np.finfo(np.float32).max)
    for sa1, sb1 in ((top / 448, top / 448), (top, top), (np.float32(2.0 ** -149), top), (0, top), (top, 0)):
        ca, cb = (rng.integers(1, 0x60, (r, ld), dtype=np.uint8) for r in (M, N))
        ca[:, :128] = 0
        sa = np.ones((kb, M), np.float32)
        sb = np.ones((kb, N) if b_scale == TILE else ((N + 127) // 128, kb), np.float32)
        sa[0] = sa1
        if b_scale == TILE:
            sb[0] = sb1
        else:
            sb[:, 0] = sb1
        va, vb = (q8.e4m3_decode(c[:, 128:K]) for c in (ca, cb))
        for ct in (BF, F32):
            name = f"zeros {M}x{N}x{K} {sa1} {sb1} b_scale={b_scale} c={ct}"
            print("[case]", name, flush=True)
            c = torch.full((M, N), np.nan, dtype=DT[ct], device="cuda")
            d = moe.make_block_mm_desc(M, N, K, b_scale=b_scale, c_type=ct)
            scratch = torch.full((max(1, moe.moe_block_mm_scratch_bytes(d)),), 0xA5, dtype=torch.uint8, device="cuda")
            assert moe.moe_block_mm(d, *[torch.from_numpy(v).cuda() for v in (ca, sa, cb, sb)], c, scratch) == moe.MOE_OK
            torch.cuda.synchronize()
            _check(c, va, vb, K, ct, name)


@pytest.mark.parametrize("t", [BF, F32])
def test_values_and_weights_of_any_size(t):
    """The same through the quantisers: values near 2^-70 against weights near 2^-65, and 2^75 against 2^-140."""
    rng = np.random.default_rng(1)
    for M, N, K in ((1, 64, 300), (20, 33, 1000), (500, 260, 384)):
        for ea, eb in ((-62, -60), (75, -140), (100, -120)):
            print(f"[case] values {M}x{N}x{K} 2^{ea} 2^{eb} type={t}", flush=True)
            x = torch.from_numpy((rng.uniform(1, 2, (M, K)) * 2.0 ** ea).astype(np.float32)).to(DT[t]).cuda()
            w = torch.from_numpy((rng.uniform(1, 2, (N, K)) * 2.0 ** eb).astype(np.float32)).cuda()
            ld, kb, nb = (K + 15) // 16 * 16, (K + 127) // 128, (N + 127) // 128
            new = lambda *s, u=torch.float32: torch.empty(s, dtype=u, device="cuda")  # noqa: E731
            wq, ws, xq, xs = new(N, ld, u=torch.uint8), new(nb, kb), new(M, ld, u=torch.uint8), new(kb, M)
            moe.check(moe.moe_block_quant(moe.make_block_quant_desc(N, K, F32, BLOCK), w, wq, ws))
            moe.check(moe.moe_block_quant(moe.make_block_quant_desc(M, K, t), x, xq, xs))
            c = torch.full((M, N), np.nan, device="cuda")
            d = moe.make_block_mm_desc(M, N, K, a_type=t, c_type=F32)
            scratch = torch.full((max(1, moe.moe_block_mm_scratch_bytes(d)),), 0xA5, dtype=torch.uint8, device="cuda")
            assert moe.moe_block_mm(d, x, None, wq, ws, c, scratch) == moe.MOE_OK
            torch.cuda.synchronize()
            va = q8.e4m3_decode(xq.cpu().numpy()[:, :K]) * _wide(xs.cpu().numpy().T, K, 1)
            vb = q8.e4m3_decode(wq.cpu().numpy()[:, :K]) * _wide(_wide(ws.cpu().numpy(), N, 0), K, 1)
            _check(c, va, vb, K, F32, "values")


@pytest.mark.parametrize("M,N,K", [(3, 40, 300), (2000, 900, 300), (700, 256, 520), (1500, 1900, 300), (2040, 2000, 520),
                                   (2890, 2900, 300)])
@pytest.mark.parametrize("b_scale", [TILE, BLOCK])
def test_large_products_that_cancel(M, N, K, b_scale):
    """A run's products may pass fp32's range once scaled where their sum does not: 448^2 and -448^2 beside
    terms of 1, which leave their number, under scales whose product is up to 2^119 (448^2 2^119 = 2^136)."""
    kb, ld = (K + 127) // 128, (K + 15) // 16 * 16
    av, bv = np.ones((M, K)), np.ones((N, K))
    av[:, ::16], bv[:, ::16] = 448, 448
    av[:, 1::16], bv[:, 1::16] = 448, -448
    if K % 16 == 1:
        av[:, K - 1] = bv[:, K - 1] = 1
    pad = lambda c: np.pad(q8.e4m3_encode(c), ((0, 0), (0, ld - K)))  # noqa: E731
    for ea, eb in ((60, 59), (119, -3), (110, 9), (-20, 119), (100, -140), (52, 51)):
        sa = np.full((kb, M), 2.0 ** ea, np.float32)
        sb = np.full((kb, N) if b_scale == TILE else ((N + 127) // 128, kb), 2.0 ** eb, np.float32)
        ref = np.float64((av[:1] @ bv[:1].T).item()) * 2.0 ** (ea + eb)
        assert ref < 2.0 ** 128
        for ct in (BF, F32):
            print(f"[case] cancel {M}x{N}x{K} 2^{ea} 2^{eb} b_scale={b_scale} c={ct}", flush=True)
            c = torch.full((M, N), np.nan, dtype=DT[ct], device="cuda")
            d = moe.make_block_mm_desc(M, N, K, b_scale=b_scale, c_type=ct)
            scratch = torch.full((max(1, moe.moe_block_mm_scratch_bytes(d)),), 0xA5, dtype=torch.uint8, device="cuda")
            dev = [torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in (pad(av), sa, pad(bv), sb)]
            assert moe.moe_block_mm(d, *dev, c, scratch) == moe.MOE_OK
            torch.cuda.synchronize()
            # every partial sum is a whole number below 2^24 times a power of two: exact but for the result's rounding
            got = c.cpu().double().numpy()
            assert np.all(np.abs(got - ref) <= (2.0 ** -8 if ct == BF else U) * ref), (got.min(), got.max(), ref)
