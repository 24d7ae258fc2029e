"""Host-side checks of the operators around the layer (moe_balance_*, moe_block_*, moe_grad_*): the
documented status for every refused call.  No call here reaches a kernel launch."""
from __future__ import annotations

import ctypes

import pytest
import torch

import mixture_experts_layer_31_amd as moe

FAKE = 0x7F0000000000  # never dereferenced: every call below is refused, or does nothing
OK, EINVAL, ESCRATCH, EALIGN, EUNSUP = (moe.MOE_OK, moe.MOE_EINVAL, moe.MOE_ESCRATCH, moe.MOE_EALIGN,
                                        moe.MOE_EUNSUPPORTED)


def _bal_fwd(d, z=FAKE, idx=FAKE, valid=None, counts=FAKE, mp=FAKE, losses=FAKE, scratch=FAKE, n=1 << 30):
    return moe.lib().moe_balance_fwd(ctypes.byref(d), z, idx, valid, counts, mp, losses, scratch, n, None)


def _bal_bwd(d, z=FAKE, valid=None, counts=FAKE, dl=FAKE, idx=None, w=None, dw=None, dz=FAKE + 4096):
    return moe.lib().moe_balance_bwd(ctypes.byref(d), z, valid, counts, dl, idx, w, dw, dz, None)


def test_balance_refusals():
    ok = moe.make_desc(64, 0, 0, 128, 8)
    need = moe.moe_balance_scratch_bytes(ok)
    assert need >= 128 * 8
    for bad, code in ((moe.make_desc(-1, 0, 0, 128, 8), EINVAL), (moe.make_desc(64, 0, 0, 0, 8), EINVAL),
                      (moe.make_desc(64, 0, 0, 8, 9), EINVAL), (moe.make_desc(64, 0, 0, 8, 0), EINVAL),
                      (moe.make_desc(1 << 28, 0, 0, 8, 8), EINVAL),
                      (moe.make_desc(64, 0, 0, 1025, 8), EUNSUP)):
        assert _bal_fwd(bad) == code and _bal_bwd(bad) == code
        assert moe.moe_balance_scratch_bytes(bad) == 0
    for k in ("z", "idx", "counts", "mp", "losses", "scratch"):
        assert _bal_fwd(ok, **{k: None}) == EINVAL, k
        assert _bal_fwd(ok, **{k: FAKE + 2}) == EALIGN, k
    assert _bal_fwd(ok, scratch=FAKE + 8) == EALIGN
    assert _bal_fwd(ok, n=need - 1) == ESCRATCH
    for k in ("z", "counts", "dl", "dz"):
        assert _bal_bwd(ok, **{k: None}) == EINVAL, k
        assert _bal_bwd(ok, **{k: FAKE + 2}) == EALIGN, k
    assert _bal_bwd(ok, dz=FAKE) == EINVAL  # dlogits over the logits
    far = FAKE + (1 << 30)
    for at, k in ((far, "z"), (far + 64 * 128 * 4 - 4, "counts"), (far - 4, "dl"), (far - 8, "valid"), (far - 64 * 8 * 4 + 4, "idx")):
        parts = dict(idx=FAKE + (1 << 20), w=FAKE + (1 << 20), dw=FAKE + (1 << 20))
        assert _bal_bwd(ok, **{**parts, "dz": far, k: at}) == EINVAL, k
    for part in (dict(idx=FAKE), dict(idx=FAKE, w=FAKE), dict(w=FAKE, dw=FAKE)):
        assert _bal_bwd(ok, **part) == EINVAL, part
    assert _bal_bwd(ok, idx=FAKE, w=FAKE + 1, dw=FAKE) == EALIGN
    assert _bal_bwd(moe.make_desc(64, 0, 0, 128, 65), idx=FAKE, w=FAKE, dw=FAKE) == EUNSUP
    assert moe.lib().moe_balance_fwd(None, *[FAKE] * 7, 1 << 30, None) == EINVAL
    # no tokens: nothing to write a gradient to
    assert _bal_bwd(moe.make_desc(0, 0, 0, 128, 8), None, None, None, None, dz=None) == OK


def _quant(q, x=FAKE, codes=FAKE, scales=FAKE, codes_t=None, scales_t=None):
    return moe.lib().moe_block_quant(ctypes.byref(q), x, codes, scales, codes_t, scales_t, None)


def test_block_quant_refusals():
    mk = moe.make_block_quant_desc
    ok = mk(100, 200)
    assert (ok.ld_in, ok.ld_codes, ok.ld_codes_t) == (200, 208, 112)
    for bad in (mk(-1, 200), mk(100, -1), mk(100, 200, in_type=moe.MOE_TYPE_E4M3), mk(100, 200, scale=2),
                mk(100, 200, ld_in=199), mk(100, 200, ld_codes=192)):
        assert _quant(bad) == EINVAL
    assert _quant(mk(100, 200, ld_codes_t=96), codes_t=FAKE, scales_t=FAKE) == EINVAL
    for part in (dict(x=None), dict(codes=None), dict(scales=None), dict(codes=None, scales=None),
                 dict(codes_t=FAKE), dict(scales_t=FAKE)):
        assert _quant(ok, **part) == EINVAL, part
    for part in (dict(x=FAKE + 1), dict(codes=FAKE + 8), dict(scales=FAKE + 2),
                 dict(codes_t=FAKE + 4, scales_t=FAKE), dict(codes_t=FAKE, scales_t=FAKE + 1)):
        assert _quant(ok, **part) == EALIGN, part
    assert _quant(mk(100, 200, ld_codes=216)) == EALIGN
    assert _quant(mk(100, 200, ld_codes=1 << 22)) == EUNSUP
    assert _quant(mk(2 ** 31 - 1, 2 ** 31 - 1, ld_codes=2 ** 31)) == EUNSUP
    assert moe.lib().moe_block_quant(None, *[FAKE] * 5, None) == EINVAL
    for r, c in ((0, 200), (100, 0)):
        assert _quant(mk(r, c), x=None) == OK


def _mm(m, a=FAKE, sa=FAKE, b=FAKE, sb=FAKE, c=FAKE, scratch=None, n=0):
    return moe.lib().moe_block_mm(ctypes.byref(m), a, sa, b, sb, c, scratch, n, None)


def test_block_quant_limits():
    mk = moe.make_block_quant_desc
    assert _quant(mk(2 ** 31 - 1, 1)) == EUNSUP
    assert _quant(mk(1, 2 ** 31 - 1), codes=None, scales=None, codes_t=FAKE, scales_t=FAKE) == EUNSUP
    assert _quant(mk(4096, 4096, ld_in=1 << 40)) == EUNSUP


def test_block_mm_limits():
    mk = moe.make_block_mm_desc
    assert _mm(mk(2 ** 28, 2 ** 16, 16), n=0) == EUNSUP  # 2^32 tiles of 64 x 64 or more
    big = mk(2 ** 28, 64, 16, a_type=moe.MOE_TYPE_BF16)
    assert _mm(big, sa=None, scratch=FAKE, n=1 << 62) == EUNSUP and moe.moe_block_mm_scratch_bytes(big) == 0


def test_block_mm_refusals():
    mk = moe.make_block_mm_desc
    ok = mk(64, 48, 200)
    for bad in (mk(-1, 48, 200), mk(64, -1, 200), mk(64, 48, -1), mk(64, 48, 200, a_type=3),
                mk(64, 48, 200, b_scale=2), mk(64, 48, 200, c_type=moe.MOE_TYPE_E4M3),
                mk(64, 48, 200, flags=2), mk(64, 48, 200, flags=moe.MOE_MM_ACCUMULATE),
                mk(64, 48, 200, lda=192), mk(64, 48, 200, ldb=192), mk(64, 48, 200, ldc=47)):
        assert _mm(bad) == EINVAL
        assert moe.moe_block_mm_scratch_bytes(bad) == 0
    for k in ("a", "sa", "b", "sb", "c"):
        assert _mm(ok, **{k: None}) == EINVAL, k
    for part in (dict(a=FAKE + 8), dict(b=FAKE + 8), dict(sa=FAKE + 2), dict(sb=FAKE + 2), dict(c=FAKE + 1)):
        assert _mm(ok, **part) == EALIGN, part
    assert _mm(mk(64, 48, 200, lda=200)) == EALIGN
    assert _mm(mk(64, 48, 200, ldb=216)) == EALIGN
    assert _mm(mk(64, 48, 200, lda=1 << 22)) == EUNSUP
    assert _mm(mk(64, 48, 200, ldb=1 << 22)) == EUNSUP
    # scales past 2^31 bytes
    assert _mm(mk(2 ** 31 - 1, 16, 200)) == EUNSUP
    # values as they are: scratch for their codes, and no scales
    raw = mk(64, 48, 200, a_type=moe.MOE_TYPE_BF16)
    need = moe.moe_block_mm_scratch_bytes(raw)
    assert need >= 64 * 208 + 2 * 64 * 4
    assert _mm(raw, scratch=FAKE, n=need) == EINVAL  # a_scales given
    assert _mm(raw, sa=None, scratch=FAKE, n=need - 1) == ESCRATCH
    assert _mm(raw, sa=None, scratch=None, n=need) == EINVAL
    assert _mm(raw, sa=None, scratch=FAKE + 8, n=need) == EALIGN
    assert _mm(raw, sa=None, a=FAKE + 1, scratch=FAKE, n=need) == EALIGN
    assert moe.lib().moe_block_mm(None, *[FAKE] * 6, 0, None) == EINVAL
    for m in (mk(0, 48, 200), mk(64, 0, 200)):
        assert _mm(m, None, None, None, None, None) == OK
    # nothing to add
    assert _mm(mk(64, 48, 0, c_type=moe.MOE_TYPE_F32, flags=moe.MOE_MM_ACCUMULATE), None, None, None, None) == OK


def _list(*entries):
    return (moe.moe_grad * len(entries))(*[moe.moe_grad(*e) for e in entries])


def _norm(g, n=None, norm=FAKE, scratch=FAKE, nbytes=1 << 30):
    return moe.lib().moe_grad_norm(g, len(g) if n is None else n, norm, scratch, nbytes, None)


def _clip(g, n=None, norm=FAKE, max_norm=1.0):
    return moe.lib().moe_grad_clip(g, len(g) if n is None else n, norm, max_norm, None)


F32, BF16 = moe.MOE_TYPE_F32, moe.MOE_TYPE_BF16


def test_grad_list_refusals():
    good = (FAKE, FAKE, 100, F32, 0)
    for bad in ((None, FAKE, 100, F32, 0), (FAKE, FAKE, -1, F32, 0), (FAKE, FAKE, 100, 2, 0),
                (FAKE, FAKE, 100, -1, 0), (FAKE, FAKE, 100, F32, 1)):
        g = _list(good, bad)
        assert _norm(g) == EINVAL and _clip(g) == EINVAL, bad
    assert _norm(_list((FAKE + 2, FAKE, 100, F32, 0))) == EALIGN
    assert _norm(_list((FAKE + 1, FAKE, 100, BF16, 0))) == EALIGN
    assert _clip(_list((FAKE, FAKE + 4096 + 2, 100, F32, 0))) == EALIGN
    assert _norm(_list((FAKE, FAKE, 1 << 34, BF16, 0))) == EUNSUP
    assert _clip(_list((FAKE, None, 100, F32, 0))) == EINVAL
    g = _list(good)
    assert _norm(g, n=-1) == EINVAL and _clip(g, n=-1) == EINVAL
    assert _norm(None, n=1) == EINVAL and _clip(None, n=1) == EINVAL
    assert _norm(g, norm=None) == EINVAL and _norm(g, scratch=None) == EINVAL and _clip(g, norm=None) == EINVAL
    assert _norm(g, norm=FAKE + 2) == EALIGN and _norm(g, scratch=FAKE + 8) == EALIGN
    assert _clip(g, norm=FAKE + 2) == EALIGN
    assert _norm(g, nbytes=moe.moe_grad_scratch_bytes(1) - 1) == ESCRATCH
    assert moe.moe_grad_scratch_bytes(-1) == 0
    for m in (-1.0, float("nan"), float("inf")):
        assert _clip(g, max_norm=m) == EINVAL
    # nothing to scale
    assert _clip(_list(), norm=FAKE) == OK
    assert _clip(_list((None, None, 0, F32, 0)), norm=FAKE) == OK


def test_overlapping_destinations_are_refused():
    a, b = FAKE, FAKE + 400
    overlapping = (
        [(a, b, 100, F32, 0), (a, b, 100, F32, 0)],               # one dst twice
        [(a, a, 100, F32, 0), (a, a, 100, F32, 0)],               # one gradient twice, in place
        [(a, a + 4, 100, F32, 0)],                                # shifted onto itself
        [(a, b, 100, F32, 0), (b + 396, b + 4096, 4, BF16, 0)],   # dst over another's src
        [(a, b, 100, F32, 0), (b, b, 50, F32, 0)],
        [(a, a, 100, F32, 0), (a + 396, b, 1, F32, 0)],           # reads what another writes
    )
    for e in overlapping:
        assert _clip(_list(*e), norm=a - 64) == EINVAL, e
    for norm in (b, b + 396):  # a dst over the norm
        assert _clip(_list((a, b, 100, F32, 0)), norm=norm) == EINVAL


def test_binding_refuses_tensors_that_do_not_fit():
    """Host tensors, other types and short buffers come back as MOE_EINVAL instead of being read."""
    if torch.cuda.is_available():
        pytest.skip("the fitting GPU tensors are the GPU tests'")
    with pytest.raises(ValueError):
        moe.make_grad_list([torch.zeros(4)])
    with pytest.raises(ValueError):
        moe.make_grad_list([torch.zeros(4)], [])
