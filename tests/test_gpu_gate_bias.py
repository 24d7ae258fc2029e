"""The gate with a bias that is not a number somewhere, against the float64 oracle (bounds: tests/test_gpu_gate.py).

An expert whose choice is NaN has the lowest choice, as one whose logit is -inf has."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mixture_experts_layer_31_amd as moe
from tests import test_gpu_gate as tg

pytestmark = pytest.mark.gpu
F, B = torch.float32, torch.bfloat16

# 16 lanes a token: four, eight and sixteen values a lane, whole and ragged; 64: by experts, slots, groups
SHAPES = [(64, 1, 1, 6), (128, 1, 1, 8), (256, 1, 1, 8), (100, 1, 1, 5), (3, 1, 1, 3), (96, 8, 3, 8), (256, 8, 4, 8), (160, 8, 3, 6),
          (16, 16, 5, 5), (512, 1, 1, 8), (256, 1, 1, 20), (1000, 1, 1, 7), (512, 8, 4, 8), (128, 32, 9, 9), (1024, 64, 20, 16)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    moe.lib()


@pytest.mark.parametrize("E,G,top,K", SHAPES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_nan_in_the_bias(score, E, G, top, K):
    z, bias = tg._logits(E + K, 37, E)
    if score == "softmax":
        bias = bias / E
    rng = np.random.default_rng(E)
    for share in (None, 0.3, 0.9, 1.0):  # one, some, most and all of them
        bad = bias.copy()
        if share is None:
            bad[rng.integers(E)] = np.nan
        else:
            bad[rng.random(E) < share] = np.nan
        for best in (1, 2):
            tg._check(z, bad, K, score, G, top, best, name=f"nan {share}")
        tg._check(z, bad, K, score, G, top, 2, renorm=False, t=B, pad=1, off=1, name=f"nan {share}")


@pytest.mark.parametrize("E,G,top,K", SHAPES)
def test_nan_and_infinities_in_the_bias(E, G, top, K):
    z, bias = tg._logits(E + K + 1, 21, E)
    rng = np.random.default_rng(E + 1)
    kind = rng.random(E)
    bias[kind < 0.2], bias[kind > 0.8], bias[(kind > 0.5) & (kind < 0.6)] = np.nan, -np.inf, np.inf
    z[::5, ::3] = -np.inf
    for best in (1, 2):
        tg._check(z, bias, K, "sigmoid", G, top, best, name="nan and infinities")


@pytest.mark.parametrize("E,G,top,K", [(128, 1, 1, 8), (256, 8, 4, 8), (512, 1, 1, 8), (512, 8, 4, 8)])
def test_a_token_alone_and_among_others(E, G, top, K):
    """The same ids and weights whatever stands beside a token, with a NaN in the bias."""
    z, bias = tg._logits(5, 24, E)
    bias[[1, E // 2, E - 1]] = np.nan
    z[::5, ::3] = -np.inf
    zt, bt = torch.from_numpy(z).cuda(), torch.from_numpy(np.float32(bias)).cuda()
    for score in tg.SCORE:
        outs = []
        for rows in [range(0, 24), *[range(t, t + 1) for t in range(24)]]:
            n = len(rows)
            d = moe.make_gate_desc(n, E, K, tg.SCORE[score], G, top, 2)
            it, w = torch.full((n, K), -7, dtype=torch.int32, device="cuda"), torch.full((n, K), 7.0, device="cuda")
            assert moe.moe_gate_fwd(d, zt[rows.start:rows.stop], bt, it, w) == moe.MOE_OK
            outs.append((it, w))
        alone = [torch.cat(v) for v in zip(*outs[1:])]
        for got, want in zip(alone, outs[0]):
            assert torch.equal(got.view(torch.int32), want.view(torch.int32)), score
