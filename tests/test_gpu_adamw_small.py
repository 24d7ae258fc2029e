"""AdamW on the GPU where moments, scales and eps leave fp32's normal numbers.

States: the oracle's codes and scales, bit for bit (tests/test_gpu_adamw.py, whose bounds hold here too).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mixture_experts_layer_31_amd as moe
from oracle import adamw_oracle as ao
from tests import test_gpu_adamw as ta

pytestmark = pytest.mark.gpu
F, B = torch.float32, torch.bfloat16
ULP = 2.0 ** -149


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    moe.lib()


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("n", [128, 300, 2048 + 130])
def test_runs_of_subnormal_moments(t, n):
    """Runs whose largest value is 1 to 700 of the smallest numbers, with zeros of either sign in them: the scale of some
    rounds to 0."""
    for amax in (1, 2, 100, 223, 224, 225, 300, 447, 448, 449, 671, 672, 673, 700):
        rng = np.random.default_rng(amax)
        g = torch.Generator().manual_seed(amax)
        p = ta.Param(g, n, t, F, False, True, 1, 0.1, fresh=True)
        k = rng.integers(-amax, amax + 1, n)
        k[::128] = amax
        k[1::7] = 0
        p.g.copy_(torch.from_numpy(k.astype(np.float32) * np.float32(ULP)))
        assert int((p.g != 0).sum()) == int((k != 0).sum())
        ta._run([p], t=1, beta=(0.0, 0.95), name=f"of {amax} smallest numbers")  # m = g
        codes = p.m.cpu().numpy()
        assert not np.any((codes & 0x7F) == 0x7F)
        assert np.isfinite(ao.decode(codes, p.ms.cpu().numpy())).all()
        p.g.zero_()
        for step in range(2, 5):  # from what the step before left
            ta._run([p], t=step, name="after")
        assert torch.isfinite(p.p).all()


@pytest.mark.parametrize("master", [False, True])
def test_a_thousand_steps_without_a_gradient(master):
    """An expert that gets no tokens: after each hundred steps the states are those of the definition, and the
    parameter is a number throughout."""
    print(f"[case] adamw without a gradient master={master}", flush=True)
    g = torch.Generator().manual_seed(1)
    n = 64 * 128 + 77
    p = ta.Param(g, n, B, B, master, True, 0, 0.0, gstd=1e-3)
    p.g.zero_()
    p.m[5::128] = 0
    m, v = ((p.m.cpu().numpy(), p.ms.cpu().numpy()), (p.v.cpu().numpy(), p.vs.cpu().numpy()))
    d, lst = moe.make_adamw_desc(*ta.BETA, ta.EPS, moe.MOE_TYPE_E4M3), ta._list([p])
    lr, step = torch.tensor([1e-3], device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    zero = np.zeros(n, np.float32)
    for t in range(1, 1001):
        step += 1
        assert moe.moe_adamw(d, lst, lr, step) == moe.MOE_OK
        root = ao.decode(*v)
        m32, v32 = ao.moments32(zero, ao.decode(*m), root * root, *ta.BETA)
        m, v = ao.encode(m32), ao.encode(np.sqrt(v32), least=True)
        if t % 100 == 0:
            print(f"[case] step {t}", flush=True)
            for got, want in zip((p.m, p.ms, p.v, p.vs), (*m, *v)):
                assert np.array_equal(got.cpu().numpy(), want), t
            assert torch.isfinite(p.p).all() and (not master or torch.isfinite(p.master).all())
    assert np.abs(m32).max() < 1e-40


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("eps", [1e-39, 1e-42, ULP])
def test_an_eps_below_the_normal_numbers(eps, codes):
    """A parameter that has never seen a gradient moves by its decay alone: 0 / eps is 0."""
    g = torch.Generator().manual_seed(2)
    ps = [ta.Param(g, n, t, F, False, codes, 1, 0.1, fresh=True, gstd=1e-2) for n, t in ((700, F), (300, B))]
    for p in ps:
        p.g[::3] = 0
    for t in (1, 2):
        ta._run(ps, t=t, eps=eps, name=f"eps={eps}")
    assert all(torch.isfinite(p.p).all() for p in ps)
