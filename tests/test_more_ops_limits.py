"""Host-side limits of the gate, the block norms and AdamW (moe_gate_*, moe_norm_*, moe_adamw).  No call here reaches a kernel launch."""
from __future__ import annotations

import ctypes

import pytest
import torch

import mixture_experts_layer_31_amd as moe

FAKE = 0x7F0000000000  # never dereferenced: every call below is refused
MB = 1 << 20


def _at(k):
    return FAKE + k * 64 * MB


def _norm_fwd(d, b=_at(0), r=_at(1), gate=None, wp=None, w=_at(2), h=_at(3), y=_at(4)):
    return moe.lib().moe_norm_fwd(ctypes.byref(d), b, r, gate, wp, w, h, y, None)


def _norm_bwd(d, b=_at(0), h=_at(1), gate=None, wp=None, w=_at(2), dy=_at(3), dh=_at(4), db=_at(5), dr=_at(6),
              dgate=None, dwp=None, dw=_at(7), scratch=_at(8), n=1 << 30):
    return moe.lib().moe_norm_bwd(ctypes.byref(d), b, h, gate, wp, w, dy, dh, db, dr, dgate, dwp, dw, scratch, n, None)


def test_norm_in_place_is_the_residual_alone():
    """With h = r, or dr = dh, another input at the same address is still one that a written buffer lies over."""
    for kw in (dict(), dict(io_type=moe.MOE_TYPE_F32), dict(ld_b=70)):
        d = moe.make_norm_desc(4, 64, **kw)
        for k in ("b", "w", "wp", "gate"):
            assert _norm_fwd(d, h=_at(1), **{k: _at(1)}) == moe.MOE_EINVAL, (kw, k)
        for k in ("b", "h", "w", "dy"):
            assert _norm_bwd(d, dr=_at(4), **{k: _at(4)}) == moe.MOE_EINVAL, (kw, k)
        assert _norm_bwd(d, dr=_at(4), wp=_at(4), dwp=_at(9)) == moe.MOE_EINVAL
        assert _norm_bwd(d, dr=_at(4), gate=_at(4), dgate=_at(9)) == moe.MOE_EINVAL


def test_gate_tokens():
    """2^24 workgroups of 256 threads are more than a launch counts: 2^26 - 4 tokens of 64 lanes are the most."""
    for T in ((1 << 26) - 3, (1 << 26) - 1, 1 << 26):
        for E, K in ((512, 8), (8, 2)):
            d = moe.make_gate_desc(T, E, K)
            assert moe.lib().moe_gate_fwd(ctypes.byref(d), _at(0), None, _at(1 << 20), _at(2 << 20), None) == moe.MOE_EUNSUPPORTED
            assert moe.lib().moe_gate_bwd(ctypes.byref(d), _at(0), _at(1 << 20), _at(2 << 20), _at(3 << 20), None) == moe.MOE_EUNSUPPORTED
    d = moe.make_gate_desc((1 << 26) - 4, 8, 2)  # refused for its alignment, not for its size
    assert moe.lib().moe_gate_fwd(ctypes.byref(d), _at(0) + 2, None, _at(1 << 20), _at(2 << 20), None) == moe.MOE_EALIGN


def test_adamw_list_without_states():
    """A state or a scale that is missing is refused as a gradient is."""
    x = torch.zeros(200)
    u8 = torch.zeros(200, dtype=torch.uint8)
    for args in (dict(m=[None], v=[x]), dict(m=[x], v=[None]), dict(m=[u8], v=[u8], m_scales=[None], v_scales=[x]),
                 dict(m=[u8], v=[u8], m_scales=[x], v_scales=[None])):
        with pytest.raises(ValueError):
            moe.make_adamw_list([x], [x], **args)
