"""Blockwise FP8 of rows so small that their scale lies below fp32's normal numbers and its reciprocal is infinite: tokens of
values near 2^-130 and routing weights near 0.  Codes are the oracle's bit for bit; the layer stays within the bound
of tests/test_gpu_fp8.py against the oracle of the same recipe."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mixture_experts_layer_31_amd as moe
import moe_inputs as mi
from oracle import fp8_layer_oracle as fl
from tests import test_gpu_fp8 as t8
from tests.layer_harness import Layer, rel_err

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    moe.lib()


def _small(a, rows, power):
    a = a.copy()
    a[rows] = mi.bf16_round((a[rows] * np.float32(2.0 ** power)).astype(np.float32))
    return a


@pytest.mark.parametrize("name", ["fp8bwd_small", "mxfp8_small", "fp8_small"])
@pytest.mark.parametrize("power", [-118, -128])
def test_tokens_and_weights_near_nothing(name, power):
    cfg = mi.CONFIGS[name]
    inp = mi.make_inputs(cfg)
    w = inp["topk_w"].copy()
    w[::3, 1] *= np.float32(2.0 ** power)
    some = slice(1, None, 4)
    inp = dict(inp, topk_w=w, x=_small(inp["x"], some, power), dy=_small(inp["dy"], some, power))
    print(f"[case] recipe {name} with values near 2^{power}", flush=True)
    L = Layer(cfg, inp)
    L.prepare()
    L.fwd()
    torch.cuda.synchronize()
    assert L.check() == moe.MOE_OK
    if cfg.mode == mi.MODE_FP8:
        xp = inp["x"][L.routing()["src"] // cfg.K]
        t8._check_rows(L, xp, False)
    L.bwd()
    torch.cuda.synchronize()
    assert L.check() == moe.MOE_OK
    out = L.outputs()
    for k in ("y", "dx", "dw1", "dw2", "dprob"):
        assert np.isfinite(out[k]).all(), k
    ref = fl.layer(t8.RECIPE[cfg.mode], inp["x"], inp["topk_idx"], w, inp["dy"], inp["w1"], inp["w2"])
    errs = {k: rel_err(out[k], ref[k]) for k in ("y", "dx", "dw1", "dw2", "dprob")}
    print(name, power, {k: round(v, 4) for k, v in errs.items()}, flush=True)
    for k, e in errs.items():
        assert e <= t8.TOL_RECIPE, (k, e)
