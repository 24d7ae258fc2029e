"""The gate where the chosen scores lie at the end of 64-bit numbers, against the float64 oracle.

Renormalised weights of softmax scores depend on the chosen logits alone, and those of sigmoid scores that far down
too: they are the oracle's however far the row's largest logit is.  Bounds, u = 2^-24, half a step of the type:
weights u + 2^-40 relative; gradients 3 u of their sizes and half (tests/test_gpu_gate.py); 2^-126 absolute.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mixture_experts_layer_31_amd as moe
from oracle import gate_oracle as go

pytestmark = pytest.mark.gpu
U, TINY = 2.0 ** -24, 2.0 ** -126
F, B = torch.float32, torch.bfloat16
SCORE = dict(sigmoid=moe.MOE_SCORE_SIGMOID, softmax=moe.MOE_SCORE_SOFTMAX)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    moe.lib()


def _check(z, bias, K, score, groups=1, top=1, renorm=True, t=F, name=""):
    T, E = z.shape
    print(f"[case] gate {name} T={T} E={E} K={K} {score} groups={groups}/{top} renorm={renorm} {t}", flush=True)
    d = moe.make_gate_desc(T, E, K, SCORE[score], groups, top, 2, moe.MOE_TYPE_F32 if t == F else moe.MOE_TYPE_BF16,
                           moe.MOE_GATE_RENORM if renorm else 0, 2.5)
    zt = torch.from_numpy(z).to(t).cuda()
    z = zt.float().cpu().numpy()
    bt = None if bias is None else torch.from_numpy(np.float32(bias)).cuda()
    it, w = torch.full((T, K), -7, dtype=torch.int32, device="cuda"), torch.full((T, K), np.nan, device="cuda")
    dw, dz = torch.randn(T, K, generator=torch.Generator().manual_seed(1)), torch.full((T, E), np.nan, dtype=t, device="cuda")
    assert moe.moe_gate_fwd(d, zt, bt, it, w) == moe.MOE_OK
    assert moe.moe_gate_bwd(d, zt, it, dw.cuda(), dz) == moe.MOE_OK
    torch.cuda.synchronize()
    f = go.forward(z, None if bias is None else np.float32(bias), K, score, groups, top, 2, renorm, 2.5)
    assert np.array_equal(it.cpu().numpy(), f["idx"]), name
    got = w.cpu().numpy().astype(np.float64)
    rel = 40 * U if score == "softmax" and not renorm else U + 2.0 ** -40
    assert np.all(np.abs(got - f["w"]) <= rel * f["w"] + TINY), (name, float(np.abs(got - f["w"]).max()))
    if not renorm:
        assert torch.isfinite(dz).all()
        return
    ref = go.backward(z, f["idx"], dw.numpy(), score, True, 2.5)
    v, a = f["w"] / 2.5, np.abs(dw.numpy().astype(np.float64)) * 2.5
    size = np.zeros((T, E))
    np.put_along_axis(size, f["idx"].astype(np.int64), v * (a + (v * a).sum(axis=1, keepdims=True)), axis=1)
    half = U if t == F else 2.0 ** -8
    # the oracle's dense sum for experts that are not chosen: 2^-48 of the slots' sizes times their score (as there)
    bound = 3 * U * size * (1 + half) + half * np.abs(ref) + 2.0 ** -48 * f["s"] * size.sum(axis=1, keepdims=True) + TINY
    err = np.abs(dz.float().cpu().numpy() - ref)
    assert np.all(err <= bound), (name, float((err - bound).max()))


@pytest.mark.parametrize("E,G,top,K", [(64, 1, 1, 8), (128, 8, 3, 6), (64, 1, 1, 1), (64, 1, 1, 20), (600, 1, 1, 4), (64, 32, 8, 5)])
@pytest.mark.parametrize("t", [F, B])
def test_choices_far_below_the_rows_largest_logit(t, E, G, top, K):
    """The bias keeps the experts with the large logits (the first quarter) out."""
    rng = np.random.default_rng(1)
    for down in (100.0, 640.0, 700.0, 708.0, 720.0, 744.0, 747.0, 800.0, 5000.0, 1e30):
        z = rng.standard_normal((70, E)).astype(np.float32)
        z[:, E // 4:] -= np.float32(down)
        bias = np.zeros(E)
        bias[:E // 4] = -2.0
        bias[E // 4:] = rng.permutation(E - E // 4) * 2.0 ** -12  # who is chosen where all scores are 0 in fp32
        for renorm in (True, False):
            _check(z, bias, K, "softmax", G, top, renorm, t, name=f"{down} down")


@pytest.mark.parametrize("E,G,top,K", [(64, 1, 1, 8), (128, 8, 3, 6), (64, 1, 1, 1), (64, 1, 1, 20), (600, 1, 1, 4), (64, 32, 8, 5)])
@pytest.mark.parametrize("t", [F, B])
def test_sigmoid_scores_at_the_end_of_64_bits(t, E, G, top, K):
    rng = np.random.default_rng(2)
    for down in (80.0, 600.0, 640.0, 688.0, 692.0, 700.0, 708.0, 712.0, 720.0, 735.0, 752.0, 2000.0, 1e30):
        z = (rng.standard_normal((70, E)) * (2.0 if t == F else 4.0) - down).astype(np.float32)
        for renorm in (True, False):
            _check(z, None, K, "sigmoid", G, top, renorm, t, name=f"{down} down")
            _check(z, np.arange(E) / E, K, "sigmoid", G, top, renorm, t, name=f"{down} down, by the bias")
