"""Pins of the balance-loss oracle (CPU): closed forms and finite differences."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import balance_oracle as bo
from oracle import router_oracle as ro


def _case(seed, T, E, K):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((T, E))
    return z, np.argsort(-z, axis=1, kind="stable")[:, :K], rng


def test_equal_logits_and_shares_give_one():
    T, E, K = 12, 6, 2
    idx = np.arange(T * K).reshape(T, K) % E
    f = bo.forward(np.zeros((T, E)), idx)
    assert f["counts"].tolist() == [4] * E + [T]
    np.testing.assert_allclose(f["losses"], [1.0, np.log(E) ** 2], rtol=1e-14)
    # all tokens on one expert that they are sure of: E times 1 times 1
    z = np.full((T, E), -200.0)
    z[:, 3] = 0
    f = bo.forward(z, np.full((T, 1), 3))
    np.testing.assert_allclose(f["losses"][0], E, rtol=1e-14)


@pytest.mark.parametrize("masked", [False, True])
def test_gradient_is_the_difference_quotient(masked):
    z, idx, rng = _case(1, 9, 7, 3)
    valid = rng.random(9) < 0.6 if masked else None
    dl = np.array([0.7, -0.3])
    g = bo.backward(z, idx, valid, dl)
    h = 1e-5
    for t in range(9):
        for j in range(7):
            up, down = z.copy(), z.copy()
            up[t, j] += h
            down[t, j] -= h
            num = ((bo.forward(up, idx, valid)["losses"] - bo.forward(down, idx, valid)["losses"]) @ dl) / (2 * h)
            assert abs(num - g[t, j]) <= 1e-9


def test_nothing_kept_and_ids_out_of_range():
    z, idx, _ = _case(2, 5, 4, 2)
    f = bo.forward(z, idx, np.zeros(5, bool))
    assert not f["counts"].any() and not f["losses"].any()
    assert not bo.backward(z, idx, np.zeros(5, bool), np.ones(2)).any()
    idx[0] = (-1, 4)
    assert bo.forward(z, idx)["counts"][:4].sum() == 8


def test_router_part_is_the_router_oracles():
    z, _, rng = _case(3, 11, 8, 3)
    dw = rng.standard_normal((11, 3))
    f = ro.router_forward(z.astype(np.float32), 3)
    np.testing.assert_allclose(bo.router_part(f["idx"], f["w"], dw, 8),
                               ro.router_backward(z.astype(np.float32), 3, dw, f), atol=1e-12)
