"""The residual sum and norms of rows with infinities and NaN, against the float64 oracle: the same places are numbers,
infinities and NaN whatever the types are (bounds of the numbers: tests/test_gpu_norm.py)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mixture_experts_layer_31_amd as moe
from oracle import norm_oracle as no
from tests import test_gpu_norm as tn

pytestmark = pytest.mark.gpu
U, F, B = tn.U, torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    moe.lib()


@pytest.mark.parametrize("D", [40, 128, 300, 1024, 2500, 8192])
@pytest.mark.parametrize("io", [F, B])
@pytest.mark.parametrize("res", [F, B])
@pytest.mark.parametrize("post,gated", [(False, False), (True, False), (False, True), (True, True)])
def test_infinities_in_a_row(D, io, res, post, gated):
    print(f"[case] norm infinities D={D} io={io} res={res} post={post} gate={gated}", flush=True)
    T = 8
    g = torch.Generator().manual_seed(D)
    b, r = torch.randn(T, D, generator=g).to(io), torch.randn(T, D, generator=g).to(res)
    b[1, 3], b[2, D - 1], b[3, 5], b[3, 7] = np.inf, -np.inf, np.inf, np.inf
    b[4, 0], r[5, 1], r[6, 2] = np.nan, np.inf, np.nan
    gate = torch.randn(T, generator=g) if gated else None
    if gated:
        gate[0], gate[7] = -np.inf, np.inf
    wp = 1 + 0.1 * torch.randn(D, generator=g) if post else None
    w = 1 + 0.1 * torch.randn(D, generator=g)
    cu = lambda x: None if x is None else x.cuda()  # noqa: E731
    h, y = torch.zeros(T, D, dtype=res, device="cuda"), torch.zeros(T, D, dtype=io, device="cuda")
    d = moe.make_norm_desc(T, D, tn.TYPE[io], tn.TYPE[res], scale=0.5)
    assert moe.moe_norm_fwd(d, cu(b), cu(r), cu(gate), cu(wp), cu(w), h, y) == moe.MOE_OK
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore", over="ignore"):
        f = no.forward(tn._np(b), tn._np(r), tn._np(gate), tn._np(wp), None, np.float64(np.float32(1e-6)), 0.5)
        kept = tn._np(h)
        ref = no.forward(None, kept, None, None, tn._np(w), np.float64(np.float32(1e-6)), 0.0)["y"]
        size = np.abs(tn._np(r)) + np.abs(f["h"] - tn._np(r))
    for got, want, bound in ((kept, f["h"], (tn.HALF[res] + U) * 1.01 * np.abs(f["h"]) + 32 * U * size + tn.TINY),
                             (tn._np(y), ref, (tn.HALF[io] + 24 * U) * np.abs(ref) + tn.TINY)):
        assert np.array_equal(np.isnan(got), np.isnan(want))
        inf = np.isinf(want)
        assert np.array_equal(got[inf], want[inf])
        ok = np.isfinite(want)
        assert np.all(np.abs(got[ok] - want[ok]) <= bound[ok])
    if post:  # a block's output with an infinity leaves the residual as it was, but for the infinity's place
        assert np.array_equal(kept[1, 4:], tn._np(r)[1, 4:]) and np.isnan(kept[1, 3])
