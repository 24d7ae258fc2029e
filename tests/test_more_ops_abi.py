"""Host-side checks of the gate, the block norms and AdamW (moe_gate_*, moe_norm_*, moe_adamw): the documented
status for every refused call.  No call here reaches a kernel launch."""
from __future__ import annotations

import ctypes

import pytest
import torch

import mixture_experts_layer_31_amd as moe

FAKE = 0x7F0000000000  # never dereferenced: every call below is refused, or does nothing
OK, EINVAL, ESCRATCH, EALIGN, EUNSUP = (moe.MOE_OK, moe.MOE_EINVAL, moe.MOE_ESCRATCH, moe.MOE_EALIGN,
                                        moe.MOE_EUNSUPPORTED)
F32, BF16, E4M3 = moe.MOE_TYPE_F32, moe.MOE_TYPE_BF16, moe.MOE_TYPE_E4M3
MB = 1 << 20


def _at(k):
    return FAKE + k * 64 * MB


# ---------------------------------------------------------------- gate

def _gate_fwd(d, z=_at(0), bias=None, idx=_at(1), w=_at(2)):
    return moe.lib().moe_gate_fwd(ctypes.byref(d), z, bias, idx, w, None)


def _gate_bwd(d, z=_at(0), idx=_at(1), dw=_at(2), dz=_at(3)):
    return moe.lib().moe_gate_bwd(ctypes.byref(d), z, idx, dw, dz, None)


def test_gate_descriptors():
    mk = moe.make_gate_desc
    for bad in (mk(-1, 128, 8), mk(64, 0, 1), mk(64, 8, 9), mk(64, 8, 0), mk(1 << 28, 8, 8), mk(64, 128, 8, groups=0),
                mk(64, 100, 8, groups=8), mk(64, 128, 8, groups=8, top_groups=9), mk(64, 128, 8, groups=8, top_groups=0),
                mk(64, 128, 33, groups=8, top_groups=2), mk(64, 128, 8, group_best=0), mk(64, 128, 8, group_best=3),
                mk(64, 128, 8, score=2), mk(64, 128, 8, score=-1), mk(64, 128, 8, in_type=E4M3), mk(64, 128, 8, flags=4),
                mk(64, 128, 8, scale=float("nan")), mk(64, 128, 8, scale=float("inf")), mk(64, 128, 8, ld_logits=127),
                mk(64, 128, 8, ld_dlogits=127), mk(64, 128, 8, in_type=BF16, flags=moe.MOE_GATE_ACCUMULATE)):
        assert _gate_fwd(bad) == EINVAL and _gate_bwd(bad) == EINVAL, [getattr(bad, f) for f, _ in bad._fields_]
    for bad in (mk(64, 1025, 8), mk(64, 1024, 65), mk(64, 130, 8, groups=65, top_groups=65), mk(1 << 26, 128, 8), mk(64, 128, 8, ld_logits=1 << 40),
                mk(64, 128, 8, ld_dlogits=1 << 40)):
        assert _gate_fwd(bad) == EUNSUP and _gate_bwd(bad) == EUNSUP
    assert moe.lib().moe_gate_fwd(None, FAKE, None, FAKE, FAKE, None) == EINVAL
    assert moe.lib().moe_gate_bwd(None, FAKE, FAKE, FAKE, FAKE, None) == EINVAL


def test_gate_buffers():
    d = moe.make_gate_desc(64, 128, 8)
    for k in ("z", "idx", "w"):
        assert _gate_fwd(d, **{k: None}) == EINVAL
        assert _gate_fwd(d, **{k: FAKE + 2}) == EALIGN
    assert _gate_fwd(d, bias=FAKE + 2) == EALIGN
    for k in ("z", "idx", "dw", "dz"):
        assert _gate_bwd(d, **{k: None}) == EINVAL
        assert _gate_bwd(d, **{k: FAKE + 2}) == EALIGN
    assert _gate_fwd(moe.make_gate_desc(64, 128, 8, in_type=BF16), z=FAKE + 1) == EALIGN
    # over an input, from its first to its last byte
    assert _gate_bwd(d, dz=_at(0)) == EINVAL
    assert _gate_bwd(d, dz=_at(0) + 64 * 128 * 4 - 4) == EINVAL
    assert _gate_bwd(d, dz=_at(1) - 64 * 128 * 4 + 4) == EINVAL
    assert _gate_bwd(d, dz=_at(2) + 64 * 8 * 4 - 4) == EINVAL
    for k, at in dict(idx=_at(0) + 64 * 128 * 4 - 4, w=_at(1) + 64 * 8 * 4 - 4).items():  # logits, the ids
        assert _gate_fwd(d, **{k: at}) == EINVAL
    assert _gate_fwd(d, w=_at(0) - 64 * 8 * 4 + 4) == EINVAL
    assert _gate_fwd(d, bias=_at(1) - 128 * 4 + 4) == EINVAL and _gate_fwd(d, bias=_at(2) + 64 * 8 * 4 - 4) == EINVAL
    empty = moe.make_gate_desc(0, 128, 8)
    assert _gate_fwd(empty, z=None, idx=None, w=None) == OK
    assert _gate_bwd(empty, z=None, idx=None, dw=None, dz=None) == OK


def test_gate_bias_refusals():
    f = moe.lib().moe_gate_bias
    assert f(0, FAKE, 0.1, _at(1), None) == EINVAL and f(8, None, 0.1, FAKE, None) == EINVAL
    assert f(8, FAKE, 0.1, None, None) == EINVAL and f(8, FAKE, float("inf"), _at(1), None) == EINVAL
    assert f(8, FAKE, float("nan"), _at(1), None) == EINVAL
    assert f(8, FAKE + 2, 0.1, _at(1), None) == EALIGN and f(8, FAKE, 0.1, _at(1) + 1, None) == EALIGN
    assert f(8, FAKE, 0.1, FAKE + 28, None) == EINVAL


# ---------------------------------------------------------------- norm

def _norm_fwd(d, b=_at(0), r=_at(1), gate=None, wp=None, w=_at(2), h=_at(3), y=_at(4)):
    return moe.lib().moe_norm_fwd(ctypes.byref(d), b, r, gate, wp, w, h, y, None)


def _norm_bwd(d, b=_at(0), h=_at(1), gate=None, wp=None, w=_at(2), dy=_at(3), dh=_at(4), db=_at(5), dr=_at(6),
              dgate=None, dwp=None, dw=_at(7), scratch=_at(8), n=1 << 30):
    return moe.lib().moe_norm_bwd(ctypes.byref(d), b, h, gate, wp, w, dy, dh, db, dr, dgate, dwp, dw, scratch, n, None)


def test_norm_descriptors():
    mk = moe.make_norm_desc
    for bad in (mk(-1, 64), mk(4, 0), mk(4, 64, io_type=E4M3), mk(4, 64, res_type=E4M3), mk(4, 64, w_type=E4M3),
                mk(4, 64, eps=-1e-6), mk(4, 64, eps=float("nan")), mk(4, 64, eps=float("inf")),
                mk(4, 64, scale=float("nan")), mk(4, 64, scale=float("inf")),
                *[mk(4, 64, **{k: 63}) for k in ("ld_b", "ld_r", "ld_h", "ld_y")]):
        assert _norm_fwd(bad) == EINVAL and _norm_bwd(bad) == EINVAL
        assert moe.moe_norm_scratch_bytes(bad) == 0
    for bad in (mk(4, 16385), *[mk(4, 64, **{k: 1 << 40}) for k in ("ld_b", "ld_r", "ld_h", "ld_y")]):
        assert _norm_fwd(bad) == EUNSUP and _norm_bwd(bad) == EUNSUP
        assert moe.moe_norm_scratch_bytes(bad) == 0
    assert moe.lib().moe_norm_fwd(None, *[FAKE] * 7, None) == EINVAL
    assert moe.lib().moe_norm_bwd(None, *[FAKE] * 13, 1 << 30, None) == EINVAL


def test_norm_buffers():
    d = moe.make_norm_desc(4, 64)
    for k in ("r", "h", "w", "y"):
        assert _norm_fwd(d, **{k: None}) == EINVAL, k
    assert _norm_fwd(d, b=None, gate=_at(5)) == EINVAL and _norm_fwd(d, b=None, wp=_at(5)) == EINVAL
    assert _norm_fwd(d, b=None, w=None, y=None) == EINVAL  # nothing to do
    for k in ("b", "r", "h", "y"):
        assert _norm_fwd(d, **{k: FAKE + 1}) == EALIGN, k
    for k in ("gate", "wp", "w"):
        assert _norm_fwd(d, **{k: FAKE + 2}) == EALIGN, k
    # the residual in place, but not shifted, with another stride, or over anything else
    last = 4 * 64 * 2 - 2
    for over in (dict(h=_at(0)), dict(h=_at(1) + 2), dict(y=_at(1)), dict(y=_at(3) + last), dict(h=_at(2)), dict(y=_at(0)),
                 dict(h=_at(0) + last), dict(wp=_at(4)), dict(gate=_at(3))):
        assert _norm_fwd(d, **over) == EINVAL, over
    assert _norm_fwd(moe.make_norm_desc(4, 64, ld_h=65), h=_at(1)) == EINVAL
    assert _norm_fwd(moe.make_norm_desc(0, 64), b=None, r=None, w=None, h=None, y=None) == OK


def test_norm_backward_buffers():
    d = moe.make_norm_desc(4, 64)
    assert moe.moe_norm_scratch_bytes(d) >= 2 * 64 * 4  # a row each of both weights'
    for k in ("h", "w", "db", "dr", "dw", "scratch"):
        assert _norm_bwd(d, **{k: None}) == EINVAL, k
    assert _norm_bwd(d, gate=_at(9)) == EINVAL and _norm_bwd(d, dgate=_at(9)) == EINVAL
    assert _norm_bwd(d, wp=_at(9)) == EINVAL and _norm_bwd(d, dwp=_at(9)) == EINVAL
    both = dict(gate=_at(9), dgate=_at(10))
    assert _norm_bwd(d, **both, b=None) == EINVAL and _norm_bwd(d, **both, db=None) == EINVAL
    assert _norm_bwd(d, w=None, dw=None) == EINVAL  # dy without w
    assert _norm_bwd(d, n=moe.moe_norm_scratch_bytes(d) - 1) == ESCRATCH
    for k in ("b", "h", "dy", "dh", "db", "dr"):
        assert _norm_bwd(d, **{k: FAKE + 1}) == EALIGN, k
    for k in ("w", "dw"):
        assert _norm_bwd(d, **{k: FAKE + 2}) == EALIGN, k
    assert _norm_bwd(d, scratch=FAKE + 8) == EALIGN
    for over in (dict(dr=_at(0)), dict(dr=_at(4) + 2), dict(db=_at(3)), dict(db=_at(4)), dict(dr=_at(5)), dict(dw=_at(2)),
                 dict(dw=_at(6)), dict(scratch=_at(0)), dict(dr=_at(8) + 256)):
        assert _norm_bwd(d, **over) == EINVAL, over
    assert _norm_bwd(moe.make_norm_desc(4, 64, ld_r=65), dr=_at(4)) == EINVAL


# ---------------------------------------------------------------- AdamW

def _param(k=0, n=1000, pt=F32, gt=F32, wd=0.0, reserved=0, codes=False, **kw):
    a = dict(param=_at(10 * k), master=None, grad=_at(10 * k + 2), m=_at(10 * k + 3), v=_at(10 * k + 4),
             m_scale=_at(10 * k + 5) if codes else None, v_scale=_at(10 * k + 6) if codes else None)
    a.update(kw)
    return moe.moe_adamw_param(*[a[x] for x in ("param", "master", "grad", "m", "v", "m_scale", "v_scale")], n, pt, gt,
                               wd, reserved)


def _adamw(*entries, d=None, lr=_at(90), step=_at(91), norm=None, max_norm=0.0, n=None):
    g = (moe.moe_adamw_param * len(entries))(*entries)
    d = moe.make_adamw_desc() if d is None else d
    return moe.lib().moe_adamw(ctypes.byref(d), g, len(entries) if n is None else n, lr, step, norm, max_norm, None)


def test_adamw_descriptors():
    mk, nan, inf = moe.make_adamw_desc, float("nan"), float("inf")
    for bad in (mk(beta1=1.0), mk(beta1=-0.1), mk(beta1=nan), mk(beta2=1.0), mk(beta2=-0.1), mk(beta2=nan), mk(eps=-1.0),
                mk(eps=nan), mk(eps=inf), mk(eps=1e39), mk(state_type=BF16), mk(state_type=-1)):
        assert _adamw(_param(), d=bad) == EINVAL
    odd = mk()
    odd.reserved = 1
    assert _adamw(_param(), d=odd) == EINVAL
    assert moe.lib().moe_adamw(None, None, 0, FAKE, FAKE, None, 0.0, None) == EINVAL
    assert _adamw(_param(), n=-1) == EINVAL
    d = mk()
    assert moe.lib().moe_adamw(ctypes.byref(d), None, 1, FAKE, _at(1), None, 0.0, None) == EINVAL
    for m in (-1.0, nan, inf):
        assert _adamw(_param(), norm=_at(92), max_norm=m) == EINVAL
    assert _adamw(_param(), lr=None) == EINVAL and _adamw(_param(), step=None) == EINVAL
    for k in ("lr", "step", "norm"):
        assert _adamw(_param(), **{k: FAKE + 2 * MB + 2}) == EALIGN
    assert _adamw() == OK and _adamw(_param(n=0, param=None, grad=None, m=None, v=None)) == OK


def test_adamw_entries():
    e4m3 = moe.make_adamw_desc(state_type=E4M3)
    for bad in (_param(n=-1), _param(pt=E4M3), _param(gt=E4M3), _param(reserved=1), _param(wd=float("nan")),
                _param(master=_at(1)), _param(param=None), _param(grad=None), _param(m=None), _param(v=None),
                _param(m_scale=_at(5)), _param(v_scale=_at(6))):
        assert _adamw(_param(k=3), bad) == EINVAL
    for bad in (_param(), _param(codes=True, m_scale=None), _param(codes=True, v_scale=None)):
        assert _adamw(bad, d=e4m3) == EINVAL
    assert _adamw(_param(n=1 << 34)) == EUNSUP
    for k in ("param", "grad", "m", "v"):
        assert _adamw(_param(**{k: FAKE + 3 * MB + 2})) == EALIGN, k
    assert _adamw(_param(pt=BF16, param=FAKE + 1)) == EALIGN
    assert _adamw(_param(pt=BF16, master=_at(1) + 2)) == EALIGN
    for k in ("m", "v"):
        assert _adamw(_param(codes=True, **{k: FAKE + 3 * MB + 8}), d=e4m3) == EALIGN, k
    for k in ("m_scale", "v_scale"):
        assert _adamw(_param(codes=True, **{k: FAKE + 3 * MB + 2}), d=e4m3) == EALIGN, k


def test_adamw_overlaps():
    p = _param()
    e4m3 = moe.make_adamw_desc(state_type=E4M3)
    for bad in ([p, p], [_param(grad=_at(0))], [_param(grad=_at(0) + 3996)], [_param(m=_at(4))], [_param(v=_at(0) + 4)],
                [p, _param(k=1, param=_at(0) + 3996)], [p, _param(k=1, grad=_at(3) + 3996)],
                [p, _param(k=1, pt=BF16, master=_at(4) - 3996)]):
        assert _adamw(*bad) == EINVAL
    assert _adamw(_param(codes=True, m_scale=_at(4) + 999 // 4 * 4), d=e4m3) == EINVAL
    assert _adamw(_param(codes=True, v_scale=_at(5) + 28), d=e4m3) == EINVAL
    for k in ("lr", "step", "norm"):
        assert _adamw(p, **{k: _at(0) + 3996}) == EINVAL, k


def test_binding_refuses_tensors_that_do_not_fit():
    """Host tensors, other types and short buffers are refused instead of being read."""
    if torch.cuda.is_available():
        pytest.skip("the fitting GPU tensors are the GPU tests'")
    x = torch.zeros(200)
    with pytest.raises(ValueError):
        moe.make_adamw_list([x], [x], [x], [x])
    for kw in (dict(m_scales=[x]), dict(weight_decay=[0.1, 0.2]), dict(masters=[x, x])):
        with pytest.raises(ValueError):
            moe.make_adamw_list([x], [x], [x], [x], **kw)
    with pytest.raises(ValueError):
        moe.make_adamw_list([x], [x[:100]], [x], [x])
