"""Norm and clipping of lists that go past the memory-side cache, in both types, at any alignment, into other
buffers and in place.  Tolerances as in test_gpu_clip."""
from __future__ import annotations

import pytest
import torch

import mixture_experts_layer_31_amd as moe
from tests import test_gpu_clip as tc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    moe.lib()


@pytest.mark.parametrize("shift", [0, 1, 3])
def test_long_lists(shift):
    n = 21_000_000  # 84 MB in fp32, 42 in bf16: past 144 MB in all
    tc._check([(n + 5, tc.F, 1), (n + 3, tc.F, 2), (7, tc.B, 5), (n + 1, tc.B, 3), (0, tc.F, 0), (n, tc.B, 0), (9, tc.F, 3)],
              f"long, {shift}", seed=shift, shift=shift)
