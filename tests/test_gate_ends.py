"""Pins of the gate's oracle where the chosen scores lie at the end of 64-bit numbers, by hand and by differences."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import gate_oracle as go


@pytest.mark.parametrize("down", [0.0, 700.0, 744.0, 800.0, 1e6])
def test_renormalised_weights_are_the_chosen_ones_alone(down):
    """exp(-d) and exp(-d) / 3 beside each other: 3/4 and 1/4, and the gradient v (a - sum v a), however large d is."""
    z = np.array([[0.0, -down, -down - np.log(3.0)]])
    f = go.forward(z, np.array([-3.0, 1.0, 0.5]), 2, "softmax", scale=2.0)
    assert f["idx"].tolist() == [[1, 2]] and np.allclose(f["w"], [[1.5, 0.5]], rtol=1e-9)
    dz = go.backward(z, f["idx"], [[1.0, 0.0]], "softmax", scale=2.0)
    assert np.allclose(dz, [[0.0, 0.375, -0.375]], rtol=1e-9, atol=1e-12)
    # an id twice has both slots' shares
    dz = go.backward(z, [[1, 1, 2]], [[1.0, 1.0, 0.0]], "softmax")
    v = np.array([3.0, 3.0, 1.0]) / 7
    assert np.allclose(dz, [[0.0, (v[0] + v[1]) * v[2], -(v[0] + v[1]) * v[2]]], rtol=1e-9, atol=1e-12)


@pytest.mark.parametrize("down", [50.0, 600.5, 650.0, 700.0, 720.0, 740.0])
def test_sigmoid_scores_far_down_are_exponentials(down):
    z = np.array([[-down, -down - np.log(3.0)]])
    f = go.forward(z, None, 2)
    assert f["idx"].tolist() == [[0, 1]] and np.allclose(f["w"], [[0.75, 0.25]], rtol=1e-9)
    assert np.allclose(go.backward(z, f["idx"], [[1.0, 0.0]]), [[0.1875, -0.1875]], rtol=1e-9)
    assert np.allclose(go.scores(z, "sigmoid")[0, 0], np.exp(-down), rtol=1e-12)


def test_scores_that_are_0():
    z = np.array([[-2000.0, -3000.0], [-np.inf, -np.inf]])
    for score in ("sigmoid", "softmax"):
        rows = slice(0, 2) if score == "sigmoid" else slice(1, 2)
        assert not go.forward(z[rows], None, 2, score)["w"].any()
        assert not go.backward(z[rows], [[0, 1]] * len(z[rows]), np.ones((len(z[rows]), 2)), score).any()
