"""Block-scaled e4m3 matrices and their product on the GPU (through the C ABI) against the oracles.

Codes and scales are compared bit for bit.  The product against the float64 product of the same
codes' values: with S = sum |A| |B| of an output (values, scaled) and u = 2^-24,
* the sums within a run of 128 in the matrix core: for fp32 outputs exact products and an addition each,
  128 u S; for bf16 outputs eight products at a time, each cut to a multiple of 2^-13 of the
  largest one's power of two (at most 8 * 2^-13 of that product, hence 2^-10 S over all groups),
  and then the same additions;
* the scale product, the FMA over K / 128 runs and a join of split sums add (K / 128 + 20) u S;
* the output's rounding half a step: 2^-8 (bf16) or u (fp32) relative to it; an accumulated output
  one more u.
The cut's bound is far above what normal data show (1.5e-5 relative), so a bf16 output of many values
is also held to 2^-8 in the 2-norm: its rounding is at most that in every value.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mixture_experts_layer_31_amd as moe
from oracle import block_oracle as bk
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


def _x(seed, R, C, t=BF, spread=4.0):
    """[R, C] with rows and columns of uneven size, as the type holds it."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((R, C)) * np.exp2(rng.uniform(-spread, spread, (R, 1)) + rng.uniform(-spread, spread, (1, C)))
    return torch.from_numpy(x.astype(np.float32)).to(DT[t])


def _strided(x, ld, off=0, fill=0.0):
    """x on the GPU with rows ld apart, off elements into its buffer."""
    R, C = x.shape
    buf = torch.full((R * ld + off,), fill, dtype=x.dtype, device="cuda")
    v = buf[off:off + R * ld].view(R, ld) if R else buf[off:].view(0, ld)
    v[:, :C] = x.cuda()
    return v[:, :C]


def _quant(x, scale, rows=True, cols=True, t=BF, ld=None, off=0):
    R, C = x.shape
    ld = C if ld is None else ld
    d = moe.make_block_quant_desc(R, C, t, scale, ld_in=ld, ld_codes=(C + 15) // 16 * 16 + 16,
                                  ld_codes_t=(R + 15) // 16 * 16 + 32)
    rb, cb = (R + 127) // 128, (C + 127) // 128
    code = lambda n, l: torch.full((n, l), 0x55, dtype=torch.uint8, device="cuda")  # noqa: E731
    sc = lambda *s: torch.full(s, np.nan, device="cuda")  # noqa: E731
    q = (code(R, d.ld_codes), sc(rb, cb) if scale == BLOCK else sc(cb, R)) if rows else (None, None)
    qt = (code(C, d.ld_codes_t), sc(cb, rb) if scale == BLOCK else sc(rb, C)) if cols else (None, None)
    assert moe.moe_block_quant(d, _strided(x, ld, off), *q, *qt) == moe.MOE_OK
    torch.cuda.synchronize()
    return [None if v is None else v.cpu().numpy() for v in (*q, *qt)]


def _same_codes(got, want, n):
    """Codes equal, zeros to the next multiple of 16, and nothing written behind."""
    pad = (n + 15) // 16 * 16
    assert np.array_equal(got[:, :n], want)
    assert not got[:, n:pad].any() and (got[:, pad:] == 0x55).all()


def _check_quant(x, t, name, **kw):
    R, C = x.shape
    f = x.float().numpy()
    for scale in (TILE, BLOCK):
        print(f"[case] quant {name} {R}x{C} type={t} scale={scale} {kw}", flush=True)
        q, s, qt, st = _quant(x, scale, t=t, **kw)
        if scale == TILE:
            (wq, ws), (wqt, wst) = bk.quant_tiles(f), bk.quant_tiles(f.T)
        else:
            wq, ws = bk.quant_blocks(f)
            wqt, wst = wq.T, ws.T
        if q is not None:
            _same_codes(q, wq, C)
            assert np.array_equal(s, ws)
        if qt is not None:
            _same_codes(qt, wqt, R)
            assert np.array_equal(st, wst)


@pytest.mark.parametrize("R,C", [(1, 1), (1, 128), (128, 1), (3, 17), (16, 16), (127, 129), (128, 128),
                                 (129, 127), (300, 200), (255, 384), (1000, 33)])
@pytest.mark.parametrize("t", [BF, F32])
def test_quantiser_is_bit_exact(R, C, t):
    x = _x(R * 1000 + C, R, C, t)
    x[0, 0] = 0
    _check_quant(x, t, "plain")
    _check_quant(x, t, "rows only, strided", cols=False, ld=C + 5)
    _check_quant(x, t, "columns only, unaligned", rows=False, ld=C + 8, off=3)


def test_quantiser_ties_and_ranges():
    """Quotients on the borders of two codes, zero and tiny runs, the largest values."""
    mids = np.concatenate([(q8._POS_VALUES[1:] + q8._POS_VALUES[:-1]) / 2, q8._POS_VALUES]).astype(np.float32)
    rows = []
    for s in (1.0, 0.75, 3.0, 1.17, 2.0 ** -100, 2.0 ** -126, 2.0 ** 118):
        for k in (0, 1, -1):
            r = np.zeros(256, np.float32)
            r[:253] = mids[:253] * np.float32(s)
            if k:
                r = np.nextafter(r, np.float32(np.inf if k > 0 else 0))
            r[253] = r[254] = np.float32(448) * np.float32(s)
            rows.append(r)
    tiny = np.zeros((4, 256), np.float32)
    tiny[1, :7], tiny[2, 3], tiny[3, :3] = 1e-45, 3e-43, 1e-38
    x = torch.from_numpy(np.concatenate([np.stack(rows), tiny]))
    _check_quant(x, F32, "borders")
    _check_quant(x.to(torch.bfloat16), BF, "borders")
    big = torch.full((5, 130), torch.finfo(torch.float32).max)
    _check_quant(big, F32, "largest")


def test_quantiser_of_many_values():
    rng = np.random.default_rng(11)
    bits = rng.integers(0, 1 << 32, size=(256, 1024), dtype=np.uint64).astype(np.uint32).view(np.float32)
    x = np.where(np.isfinite(bits), bits, 0).astype(np.float32)
    _check_quant(torch.from_numpy(x), F32, "all magnitudes")
    near = np.exp2(rng.uniform(-9, 9, (256, 1024))).astype(np.float32)
    _check_quant(torch.from_numpy(near), F32, "near the scale")


def test_quantiser_of_nan_and_inf():
    x = torch.ones(2, 256)
    x[0, 5], x[1, 200] = float("nan"), float("inf")
    q, s, _, _ = _quant(x, TILE, cols=False, t=F32)
    v = bk.values_tiles(q[:, :256], s)
    assert np.isnan(v[0, 5]) and np.array_equal(np.delete(v[0, :128], 5), np.ones(127, np.float64) * v[0, 0])
    assert np.isfinite(v[0]).sum() == 255 and np.isnan(v[1, 128:]).all() and np.isfinite(v[1, :128]).all()


@pytest.mark.parametrize("t", [BF, F32])
def test_infinite_scales_follow_the_definition(t):
    """x / inf: codes 0, NaN (either sign) where x is infinite; and the padding stays 0."""
    x = _x(5, 130, 140, t)
    x[3, 7], x[100, 139], x[129, 0] = float("inf"), -float("inf"), float("inf")
    f = x.float().numpy()
    with np.errstate(invalid="ignore"):
        for scale in (TILE, BLOCK):
            q, s, qt, st = _quant(x, scale, t=t)
            want = [bk.quant_tiles(f), bk.quant_tiles(f.T)] if scale == TILE else [bk.quant_blocks(f)]
            if scale == BLOCK:
                want.append((want[0][0].T, want[0][1].T))
            # inf / inf is a NaN, which the oracle's encoder does not take
            for got, sc, n, nan, (wq, ws) in ((q, s, 140, np.isinf(f), want[0]), (qt, st, 130, np.isinf(f.T), want[1])):
                assert np.array_equal(sc, ws) and np.isinf(ws).any()
                _same_codes(np.where(np.pad(nan, ((0, 0), (0, got.shape[1] - n))), 0, got), np.where(nan, 0, wq), n)
                assert np.isnan(q8.e4m3_decode(got[:, :n][nan])).all()


# ---------------------------------------------------------------- product

def _codes(seed, R, K, scale, ld_extra=16, junk=0x7F):
    """(codes on the GPU [R, ld], scales, values in float64); NaN codes behind column K."""
    x = _x(seed, R, K, F32, spread=2.0).numpy()
    c, s = (bk.quant_blocks if scale == BLOCK else bk.quant_tiles)(x)
    v = (bk.values_blocks if scale == BLOCK else bk.values_tiles)(c, s)
    ld = (K + 15) // 16 * 16 + ld_extra
    buf = np.full((R, ld), junk, np.uint8)
    buf[:, :K] = c
    return torch.from_numpy(buf).cuda(), torch.from_numpy(np.ascontiguousarray(s)).cuda(), v, ld


def _bound(va, vb, K, ref, ct):
    S = np.abs(va) @ np.abs(vb).T
    out = 2.0 ** -8 if ct == BF else U
    cut = 2.0 ** -10 if ct == BF else 0.0
    return ((128 + K / 128 + 20) * U + cut) * S + out * np.abs(ref) + 2.0 ** -126


def _check_mm(M, N, K, b_scale, ct, seed=0, add=False, ldc=None, off=0):
    print(f"[case] mm {M}x{N}x{K} b_scale={b_scale} c={ct} add={add} ldc={ldc} off={off}", flush=True)
    a, sa, va, lda = _codes(seed + 1, M, K, TILE)
    b, sb, vb, ldb = _codes(seed + 2, N, K, b_scale)
    ldc = N if ldc is None else ldc
    old = torch.randn(M, N).to(DT[ct])
    buf = torch.full((M * ldc + off,), 77.0, dtype=DT[ct], device="cuda")
    c = buf[off:].view(M, ldc)
    if add:
        c[:, :N] = old.cuda()
    d = moe.make_block_mm_desc(M, N, K, b_scale=b_scale, c_type=ct, lda=lda, ldb=ldb, ldc=ldc,
                               flags=moe.MOE_MM_ACCUMULATE if add else 0)
    scratch = torch.full((moe.moe_block_mm_scratch_bytes(d),), 0xA5, dtype=torch.uint8, device="cuda")
    assert moe.moe_block_mm(d, a, sa, b, sb, c[:, :N], scratch) == moe.MOE_OK
    torch.cuda.synchronize()
    ref = va @ vb.T
    bound = _bound(va, vb, K, ref, ct)
    if add:
        ref = ref + old.double().numpy()
        bound += U * np.abs(ref)
    got = c.cpu().double().numpy()
    err = np.abs(got[:, :N] - ref)
    assert np.all(err <= bound), float((err / np.maximum(bound, 1e-300)).max())
    assert np.linalg.norm(err) <= 2.0 ** -8 * np.linalg.norm(ref)
    assert (got[:, N:] == 77).all() and (buf[:off] == 77).all()
    return got[:, :N]


SHAPES = [(1, 1, 1), (1, 128, 128), (1, 1000, 300), (2, 16, 17), (5, 33, 129), (16, 16, 16), (17, 48, 640),
          (31, 200, 1000), (64, 64, 256), (65, 130, 384), (100, 259, 257), (128, 128, 128), (200, 640, 144),
          (257, 255, 500), (300, 513, 130), (700, 256, 2048), (513, 1100, 96)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("b_scale", [TILE, BLOCK])
def test_product(M, N, K, b_scale):
    _check_mm(M, N, K, b_scale, BF, seed=M + N + K)
    _check_mm(M, N, K, b_scale, F32, seed=M + N + K, ldc=N + 3, off=1)


@pytest.mark.parametrize("M,N,K", [(1, 64, 4096), (7, 100, 700), (150, 300, 1500), (300, 260, 128), (600, 700, 200),
                                   (2100, 1030, 130)])
def test_product_added_to_c(M, N, K):
    _check_mm(M, N, K, TILE, F32, seed=3, add=True)
    _check_mm(M, N, K, BLOCK, F32, seed=4, add=True, ldc=N + 1)


# every tile size and its edges: 64 x 64 (with and without the split over two groups), 128 x 128,
# 256 x 256 (one step and several, whole and partial last runs), and a few rows past a multiple of 256
@pytest.mark.parametrize("M,N,K", [(2000, 900, 300), (2000, 900, 128), (2000, 900, 40), (2100, 1030, 300),
                                   (1030, 2100, 1153), (2100, 1030, 1280), (1100, 1900, 520), (4100, 512, 128), (700, 256, 1040), (300, 500, 131),
                                   (2900, 2890, 256), (2900, 2890, 100), (2890, 2900, 300), (2900, 2890, 129),
                                   (2816, 2816, 1000), (8195, 2048, 128), (8195, 2050, 140)])
def test_product_of_many_tiles(M, N, K):
    _check_mm(M, N, K, BLOCK, BF, seed=5)
    _check_mm(M, N, K, TILE, BF, seed=6)
    _check_mm(M, N, K, BLOCK if K % 2 else TILE, F32, seed=6)


@pytest.mark.parametrize("M,N,K", [(64, 300, 2000), (65, 67, 16000), (200, 129, 9000), (257, 131, 16389), (300, 700, 5000),
                                   (1000, 90, 8100)])
@pytest.mark.parametrize("ct", [BF, F32])
def test_long_contraction_in_parts(M, N, K, ct):
    """Too few tiles for the chip: the contraction over a workgroup's waves, or in parts that a second
    launch joins."""
    parts = moe.moe_block_mm_scratch_bytes(moe.make_block_mm_desc(M, N, K, c_type=ct)) // (M * N * 4)
    assert parts >= 2 or K == 2000
    for b_scale in (TILE, BLOCK):
        one = _check_mm(M, N, K, b_scale, ct, ldc=N + 3, off=1, add=ct == F32)
        if ct == BF:
            assert np.array_equal(one, _check_mm(M, N, K, b_scale, ct))


@pytest.mark.parametrize("M,N,K", [(1500, 1900, 300), (1537, 1793, 1100), (1440, 2048, 256), (1441, 2047, 128)])
def test_product_of_tiles_of_96_rows(M, N, K):
    """Between a round of 128 x 128 tiles and a full chip."""
    for b_scale in (TILE, BLOCK):
        _check_mm(M, N, K, b_scale, BF, ldc=N + 5)


def test_empty_contraction():
    for ct in (BF, F32):
        c = torch.full((5, 9), 3.0, dtype=DT[ct], device="cuda")
        d = moe.make_block_mm_desc(5, 7, 0, c_type=ct, ldc=9)
        assert moe.moe_block_mm(d, None, None, None, None, c) == moe.MOE_OK
        torch.cuda.synchronize()
        assert not c[:, :7].any() and (c[:, 7:] == 3).all()


@pytest.mark.parametrize("M", [1, 3, 16, 17, 33, 64, 100, 129, 500])
@pytest.mark.parametrize("t", [BF, F32])
def test_values_give_what_their_codes_give(M, t):
    """A call that quantises A itself against moe_block_quant and the product of the codes: the same
    bits where the two take the same path, and always within the product's bound."""
    for N, K, ld, off in ((256, 512, None, 0), (90, 333, 340, 1), (1000, 100, 104, 0), (40, 4096, None, 0),
                          (24, 4097, 4099, 2), (70, 3, 5, 1), (20, 7, 7, 0)):
        print(f"[case] values M={M} N={N} K={K} type={t}", flush=True)
        x = _x(M + N, M, K, t, spread=1.0)
        b, sb, vb, ldb = _codes(2, N, K, BLOCK)
        ld = K if ld is None else ld
        d = moe.make_block_mm_desc(M, N, K, a_type=t, c_type=F32, lda=ld, ldb=ldb)
        c = torch.full((M, N), np.nan, device="cuda")
        scratch = torch.full((max(1, moe.moe_block_mm_scratch_bytes(d)),), 0xFF, dtype=torch.uint8, device="cuda")
        assert moe.moe_block_mm(d, _strided(x, ld, off, fill=np.nan), None, b, sb, c, scratch) == moe.MOE_OK
        torch.cuda.synchronize()
        va = bk.values_tiles(*bk.quant_tiles(x.float().numpy()))
        ref = va @ vb.T
        assert np.all(np.abs(c.cpu().double().numpy() - ref) <= _bound(va, vb, K, ref, F32))


def test_nan_stays_in_its_row():
    x = _x(1, 70, 300, F32)
    x[13, 250] = np.nan
    b, sb, _, ldb = _codes(2, 64, 300, BLOCK)
    for rows in (x, x[13:14], x[5:20]):
        M = rows.shape[0]
        d = moe.make_block_mm_desc(M, 64, 300, a_type=F32, c_type=F32, ldb=ldb)
        c = torch.zeros(M, 64, device="cuda")
        scratch = torch.empty(max(1, moe.moe_block_mm_scratch_bytes(d)), dtype=torch.uint8, device="cuda")
        moe.check(moe.moe_block_mm(d, rows.contiguous().cuda(), None, b, sb, c, scratch))
        torch.cuda.synchronize()
        bad = torch.isnan(rows).any(dim=1)
        assert torch.equal(torch.isnan(c).all(dim=1).cpu(), bad) and torch.equal(torch.isnan(c).any(dim=1).cpu(), bad)


@pytest.mark.parametrize("T,D,N", [(1, 256, 128), (300, 200, 130), (1000, 384, 256)])
def test_linear_and_its_gradients(T, D, N):
    """y = x W^T and both its gradients through the quantiser and the three products, against the same
    recipe in float64; and the recipe's gradient against the linear layer's own (its derivative is W):
    within the rounding of the codes, 2^-4 of each factor."""
    x, w, dy = _x(1, T, D, BF, 0.5), _x(2, N, D, BF, 0.5), _x(3, T, N, BF, 0.5)
    dev = [v.cuda() for v in (x, w, dy)]
    new = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    cdiv, ld = (lambda n: (n + 127) // 128), (lambda n: (n + 15) // 16 * 16)
    wq, ws = new(N, ld(D), t=torch.uint8), new(cdiv(N), cdiv(D))
    wt, wst = new(D, ld(N), t=torch.uint8), new(cdiv(D), cdiv(N))
    moe.check(moe.moe_block_quant(moe.make_block_quant_desc(N, D, BF, BLOCK), dev[1], wq, ws, wt, wst))
    y, dx, dw = new(T, N), new(T, D), new(N, D)
    mk = moe.make_block_mm_desc
    d = mk(T, N, D, a_type=BF, c_type=F32)
    scratch = new(max(1, moe.moe_block_mm_scratch_bytes(d), moe.moe_block_mm_scratch_bytes(mk(N, D, T, b_scale=TILE)),
                      moe.moe_block_mm_scratch_bytes(mk(T, D, N))), t=torch.uint8)
    moe.check(moe.moe_block_mm(d, dev[0], None, wq, ws, y, scratch))
    gq, gs, gt, gst = new(T, ld(N), t=torch.uint8), new(cdiv(N), T), new(N, ld(T), t=torch.uint8), new(cdiv(T), N)
    moe.check(moe.moe_block_quant(moe.make_block_quant_desc(T, N, BF), dev[2], gq, gs, gt, gst))
    xt, xst = new(D, ld(T), t=torch.uint8), new(cdiv(T), D)
    moe.check(moe.moe_block_quant(moe.make_block_quant_desc(T, D, BF), dev[0], None, None, xt, xst))
    moe.check(moe.moe_block_mm(mk(T, D, N, c_type=F32), gq, gs, wt, wst, dx, scratch))
    moe.check(moe.moe_block_mm(mk(N, D, T, b_scale=TILE, c_type=F32), gt, gst, xt, xst, dw, scratch))
    torch.cuda.synchronize()
    f = [v.double().numpy() for v in (x, w, dy)]
    tiles = lambda v: bk.values_tiles(*bk.quant_tiles(v.astype(np.float32)))  # noqa: E731
    wv = bk.values_blocks(*bk.quant_blocks(f[1].astype(np.float32)))
    for got, a, b, plain in ((y, tiles(f[0]), wv, (f[0], f[1])), (dx, tiles(f[2]), wv.T, (f[2], f[1].T)),
                             (dw, tiles(f[2].T), tiles(f[0].T), (f[2].T, f[0].T))):
        got, ref = got.cpu().double().numpy(), a @ b.T
        assert np.all(np.abs(got - ref) <= _bound(a, b, a.shape[1], ref, F32))
        # relative 2^-4 of a normal code, half its smallest step (2^-10 of a scale) below: amax / 448 / 2^10 more
        size = np.abs(plain[0]) @ np.abs(plain[1]).T
        room = 2 ** -4 * (2 + 2 ** -4) * size
        room += a.shape[1] * 2.0 ** -10 / 448 * 2 * np.abs(plain[0]).max() * np.abs(plain[1]).max() * 1.07
        assert np.all(np.abs(got - plain[0] @ plain[1].T) <= room + _bound(a, b, a.shape[1], ref, F32))


def test_same_bits_on_another_stream_and_in_graphs():
    """Two captured graphs that share a scratch buffer, replayed between eager calls."""
    runs = []
    scratch = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    for M, N, K in ((3, 700, 900), (130, 260, 1100)):
        x = _x(M, M, K).cuda()
        b, sb, _, ldb = _codes(2, N, K, BLOCK)
        d = moe.make_block_mm_desc(M, N, K, a_type=BF, ldb=ldb)
        assert moe.moe_block_mm_scratch_bytes(d) <= scratch.numel()
        c = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        call = (lambda d=d, x=x, b=b, sb=sb, c=c: moe.check(moe.moe_block_mm(d, x, None, b, sb, c, scratch)))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        side.synchronize()
        ref = c.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        runs.append((call, g, c, ref))
    for _ in range(3):
        for call, g, c, ref in runs:
            c.fill_(7)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(c, ref)
            c.fill_(7)
            call()
            torch.cuda.synchronize()
            assert torch.equal(c, ref)


def test_offsets_past_2_31_bytes():
    """Rows of C, A and B whose first element lies past 2^31 bytes of their buffers."""
    M, N, K, ldc = 600, 256, 128, 4 << 20
    a, sa, va, lda = _codes(1, M, K, TILE)
    b, sb, vb, ldb = _codes(2, N, K, BLOCK)
    wide = torch.zeros(M, (1 << 22) - 16, dtype=torch.uint8, device="cuda")
    wide[:, :K] = a[:, :K]
    c = torch.zeros(M, ldc, device="cuda")
    d = moe.make_block_mm_desc(M, N, K, c_type=F32, lda=wide.stride(0), ldb=ldb, ldc=ldc)
    scratch = torch.empty(max(1, moe.moe_block_mm_scratch_bytes(d)), dtype=torch.uint8, device="cuda")
    moe.check(moe.moe_block_mm(d, wide, sa, b, sb, c, scratch))
    torch.cuda.synchronize()
    got, ref = c[:, :N].cpu().double().numpy(), va @ vb.T
    assert np.all(np.abs(got - ref) <= _bound(va, vb, K, ref, F32))
    assert not c[:, N:N + 64].any()


@pytest.mark.parametrize("scale", [TILE, BLOCK])
def test_quantiser_offsets_past_2_32_bytes(scale):
    """Rows of x 16 MB apart, and codes 4 MB apart, against the same matrix in compact rows."""
    R, C, ld_in, ld = 600, 300, 8 << 20, (4 << 20) - 16
    print(f"[case] quant large scale={scale}", flush=True)
    x = _x(3, R, C)
    far = torch.empty(R, ld_in, dtype=torch.bfloat16, device="cuda")
    far[:, :C] = x.cuda()
    q, s, qt, st = _quant(x, scale)
    codes = torch.zeros(R, ld, dtype=torch.uint8, device="cuda")
    codes_t = torch.zeros(C, ld, dtype=torch.uint8, device="cuda")
    sc, sct = torch.empty(s.shape, device="cuda"), torch.empty(st.shape, device="cuda")
    d = moe.make_block_quant_desc(R, C, BF, scale, ld_in=ld_in, ld_codes=ld, ld_codes_t=ld)
    assert moe.moe_block_quant(d, far, codes, sc, codes_t, sct) == moe.MOE_OK
    torch.cuda.synchronize()
    assert np.array_equal(codes[:, :C].cpu().numpy(), q[:, :C]) and np.array_equal(codes_t[:, :R].cpu().numpy(), qt[:, :R])
    assert np.array_equal(sc.cpu().numpy(), s) and np.array_equal(sct.cpu().numpy(), st)
    assert not codes[:, 304:320].any() and not codes_t[:, 608:620].any()


def test_two_streams_at_once():
    """Products on two streams, each with scratch of its own."""
    jobs = []
    for M, N, K in ((300, 260, 9000), (130, 700, 5000)):
        x = _x(M, M, K).cuda()
        b, sb, _, ldb = _codes(2, N, K, BLOCK)
        d = moe.make_block_mm_desc(M, N, K, a_type=BF, ldb=ldb)
        scratch = torch.empty(moe.moe_block_mm_scratch_bytes(d), dtype=torch.uint8, device="cuda")
        jobs.append((d, x, b, sb, torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), scratch, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for d, x, b, sb, c, scratch, side in jobs:
            with torch.cuda.stream(side):
                moe.check(moe.moe_block_mm(d, x, None, b, sb, c, scratch))
    torch.cuda.synchronize()
    for d, x, b, sb, c, scratch, _ in jobs:
        got = c.clone()
        moe.check(moe.moe_block_mm(d, x, None, b, sb, c, scratch))
        torch.cuda.synchronize()
        assert torch.equal(got, c)


def test_binding_refuses_tensors_that_do_not_fit():
    d = moe.make_block_mm_desc(4, 8, 32)
    a, b = (torch.zeros(n, 32, dtype=torch.uint8, device="cuda") for n in (4, 8))
    sa, sb = torch.ones(1, 4, device="cuda"), torch.ones(1, 1, device="cuda")
    c = torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda")
    scratch = torch.zeros(max(1, moe.moe_block_mm_scratch_bytes(d)), dtype=torch.uint8, device="cuda")
    assert moe.moe_block_mm(d, a, sa, b, sb, c, scratch) == moe.MOE_OK
    for bad in ((a.cpu(), sa, b, sb, c), (a, sa, b[:7], sb, c), (a, sa, b, sb, c.float()), (a.float(), sa, b, sb, c),
                (a, sa[:, :3], b, sb, c), (torch.zeros(4, 64, dtype=torch.uint8, device="cuda"), sa, b, sb, c),
                (a, sa, torch.zeros(32, 8, dtype=torch.uint8, device="cuda").t(), sb, c)):
        assert moe.moe_block_mm(d, *bad, scratch) == moe.MOE_EINVAL
    assert moe.moe_block_mm(d, a.view(torch.float8_e4m3fn), sa, b, sb, c, scratch) == moe.MOE_OK
    v = moe.make_block_mm_desc(4, 8, 32, a_type=BF)
    x = torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda")
    room = torch.zeros(moe.moe_block_mm_scratch_bytes(v), dtype=torch.uint8)
    assert moe.moe_block_mm(v, x, None, b, sb, c, room.cuda()) == moe.MOE_OK
    for bad in (room, None):
        assert moe.moe_block_mm(v, x, None, b, sb, c, bad) == moe.MOE_EINVAL
    torch.cuda.synchronize()
