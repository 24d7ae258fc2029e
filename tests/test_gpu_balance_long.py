"""Balance loss of long batches: the sums over the tokens do not gather their roundings.

With equal logits p = 1 / E is one rounding off for every token alike (z - max = 0, its exp is 1 and
the row's sum E), so mean_p is n such values over n: in 64 bits nothing is added to that, a wave's and a
block's sum are rounded to fp32 and mean_p itself, 4 u in all with u = 2^-24.  losses[0] = sum of f with
one more rounding; lse = log E within 3 u (an ulp of logf and a rounding), its square 7 u, the mean
10 u.  An fp32 sum that adds the same number over and over instead is off by the same part of a step
each time.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mixture_experts_layer_31_amd as moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    moe.lib()


@pytest.mark.parametrize("T,E", [(256, 3), (1 << 22, 3), (1 << 22, 7), (1 << 20, 100), (1 << 18, 300), (1 << 18, 600)])
def test_equal_logits(T, E):
    print(f"[case] balance equal logits T={T} E={E}", flush=True)
    d = moe.make_desc(T, 0, 0, E, 1)
    z = torch.zeros(T, E, device="cuda")
    idx = torch.full((T, 1), E - 1, dtype=torch.int32, device="cuda")
    counts = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    mean_p, losses = torch.zeros(E, device="cuda"), torch.zeros(2, device="cuda")
    scratch = torch.empty(moe.moe_balance_scratch_bytes(d), dtype=torch.uint8, device="cuda")
    assert moe.moe_balance_fwd(d, z, idx, None, counts, mean_p, losses, scratch) == moe.MOE_OK
    torch.cuda.synchronize()
    assert counts[E - 1].item() == T and counts[E].item() == T
    p, loss = mean_p.cpu().double().numpy(), losses.cpu().double().numpy()
    assert np.abs(p * E - 1).max() <= 4 * U, float(np.abs(p * E - 1).max() / U)
    assert abs(loss[0] - 1) <= 5 * U and abs(loss[1] / np.log(E) ** 2 - 1) <= 10 * U, (loss - 1) / U
