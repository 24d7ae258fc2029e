"""Pins of the gate's, the norms' and AdamW's oracles against facts that do not come from them: hand
examples, differences, torch's autograd and its AdamW."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import adamw_oracle as ao
from oracle import gate_oracle as go
from oracle import norm_oracle as no


def test_gate_by_hand():
    # sigmoid(0) = 1/2, sigmoid(ln 3) = 3/4, sigmoid(-ln 3) = 1/4
    z = np.log(np.array([[1.0, 3.0, 1 / 3, 3.0]]))
    f = go.forward(z, None, 2)
    assert f["idx"].tolist() == [[1, 3]] and np.allclose(f["w"], [[0.5, 0.5]], rtol=1e-15)
    # the bias changes the choice and not the weights
    f = go.forward(z, np.array([0.0, 0.0, 0.75, 0.0]), 2, renorm=False, scale=2.0)
    assert f["idx"].tolist() == [[2, 1]] and np.allclose(f["w"], [[0.5, 1.5]], rtol=1e-15)
    # two groups of two: scores 1.25 and 1.0
    f = go.forward(z, None, 1, groups=2, top_groups=1)
    assert f["idx"].tolist() == [[1]]
    # by their best alone they are equal: the lower group
    f = go.forward(z, None, 2, groups=2, top_groups=1, group_best=1)
    assert f["idx"].tolist() == [[1, 0]]


def test_gate_masked_rows():
    ninf = -np.inf
    z = np.array([[ninf, 0.0, ninf, ninf], [ninf] * 4, [np.nan, 0.0, 1.0, ninf]])
    f = go.forward(z, None, 2)
    assert f["idx"].tolist() == [[1, 0], [0, 1], [2, 1]]
    assert np.allclose(f["w"][0], [1.0, 0.0]) and not f["w"][1].any()
    f = go.forward(z[:2], None, 2, score="softmax")
    assert f["idx"].tolist() == [[1, 0], [0, 1]] and not f["w"][1].any()
    # a group with one expert left is ahead of one with none
    f = go.forward(z[:1, [0, 2, 3, 1]], None, 2, groups=2, top_groups=1)
    assert f["idx"].tolist() == [[3, 2]]
    assert not go.backward(z[1:2], [[0, 1]], np.ones((1, 2))).any()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gate_gradient(score, renorm):
    rng = np.random.default_rng(1)
    T, E, K = 5, 12, 3
    z, dw = rng.standard_normal((T, E)), rng.standard_normal((T, K))
    f = go.forward(z, rng.standard_normal(E) * 0.1, K, score, 3, 2, renorm=renorm, scale=2.5)
    dz = go.backward(z, f["idx"], dw, score, renorm, 2.5)
    x = torch.tensor(z, requires_grad=True)
    s = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, 1)
    w = s.gather(1, torch.tensor(f["idx"]).long())
    w = 2.5 * (w / w.sum(1, keepdim=True) if renorm else w)
    assert np.allclose(w.detach().numpy(), f["w"], rtol=1e-13)
    (w * torch.tensor(dw)).sum().backward()
    assert np.allclose(dz, x.grad.numpy(), rtol=1e-10, atol=1e-14)
    # an id twice has both slots' gradients; one out of range none
    idx = np.array([[1, 1, 40]] * T)
    dz = go.backward(z, idx, dw, score, renorm, 2.5)
    x.grad = None
    s = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, 1)
    w = s[:, [1, 1]]
    w = 2.5 * (w / w.sum(1, keepdim=True) if renorm else w)
    (w * torch.tensor(dw[:, :2])).sum().backward()
    assert np.allclose(dz, x.grad.numpy(), rtol=1e-10, atol=1e-14)


def test_bias_step():
    got = go.bias_step([2, 4, 3, 3], 0.5, [0.0, 0.0, 1.0, -1.0])
    assert got.tolist() == [0.5, -0.5, 1.0, -1.0]
    assert go.bias_step([1, 2], 0.25, [0.0, 0.0]).tolist() == [0.25, -0.25]


@pytest.mark.parametrize("post,gated", [(False, False), (True, False), (False, True), (True, True)])
def test_norm_against_autograd(post, gated):
    rng = np.random.default_rng(2)
    T, D, eps, scale = 4, 9, 1e-3, 0.7
    leaf = {k: torch.tensor(rng.standard_normal(s), requires_grad=True)
            for k, s in dict(b=(T, D), r=(T, D), w=(D,), w_post=(D,), gate=(T,)).items()}
    dy, dh = rng.standard_normal((T, D)), rng.standard_normal((T, D))
    norm = lambda x: x * torch.rsqrt(x.square().mean(1, keepdim=True) + eps)  # noqa: E731
    u = norm(leaf["b"]) * leaf["w_post"] if post else leaf["b"]
    h = leaf["r"] + scale * (torch.sigmoid(leaf["gate"])[:, None] * u if gated else u)
    y = norm(h) * leaf["w"]
    ((y * torch.tensor(dy)).sum() + (h * torch.tensor(dh)).sum()).backward()
    v = {k: x.detach().numpy() for k, x in leaf.items()}
    gate, w_post = v["gate"] if gated else None, v["w_post"] if post else None
    f = no.forward(v["b"], v["r"], gate, w_post, v["w"], eps, scale)
    assert np.allclose(f["h"], h.detach().numpy(), rtol=1e-13) and np.allclose(f["y"], y.detach().numpy(), rtol=1e-12)
    g = no.backward(v["b"], f["h"], gate, w_post, v["w"], dy, dh, eps, scale)
    for k, want in leaf.items():
        if want.grad is not None:
            assert np.allclose(g["d" + k], want.grad.numpy(), rtol=1e-10, atol=1e-12), k
            assert np.all(np.abs(g["d" + k]) <= g["size"]["d" + k] * (1 + 1e-12)), k


def test_norm_gradient_by_differences():
    rng = np.random.default_rng(3)
    b, r, dy = (rng.standard_normal((2, 5)) for _ in range(3))
    gate, wp, w = rng.standard_normal(2), rng.standard_normal(5), rng.standard_normal(5)

    def loss(b, gate, wp):
        return (no.forward(b, r, gate, wp, w, 1e-2, 1.3)["y"] * dy).sum()

    h = no.forward(b, r, gate, wp, w, 1e-2, 1.3)["h"]
    g = no.backward(b, h, gate, wp, w, dy, None, 1e-2, 1.3)
    step = 1e-6
    for k, x in (("db", b), ("dgate", gate), ("dw_post", wp)):
        for i in np.ndindex(x.shape):
            at = {"db": [b, gate, wp], "dgate": [b, gate, wp], "dw_post": [b, gate, wp]}[k]
            n = ["db", "dgate", "dw_post"].index(k)
            lo, hi = x.copy(), x.copy()
            lo[i] -= step
            hi[i] += step
            d = (loss(*[hi if j == n else a for j, a in enumerate(at)])
                 - loss(*[lo if j == n else a for j, a in enumerate(at)])) / (2 * step)
            assert abs(d - g[k][i]) <= 1e-7, (k, i)


def test_adamw_against_torch():
    rng = np.random.default_rng(4)
    p0, g = rng.standard_normal(50), rng.standard_normal((3, 50))
    p = torch.tensor(p0, requires_grad=True)
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1, foreach=False)
    q, m, v = p0, np.zeros(50), np.zeros(50)
    for t in range(3):
        p.grad = torch.tensor(g[t])
        opt.step()
        q, m, v = ao.step(q, g[t], m, v, 1e-2, t + 1, 0.9, 0.95, 1e-8, 0.1)
        assert np.allclose(q, p.detach().numpy(), rtol=1e-12)
    # clipped by half, and by a norm that says nothing
    a = ao.step(p0, g[0], m, v, 1e-2, 4, 0.9, 0.95, 1e-8, 0.1, norm=4.0, max_norm=2.0)
    b = ao.step(p0, g[0] / 2, m, v, 1e-2, 4, 0.9, 0.95, 1e-8, 0.1)
    assert all(np.allclose(x, y, rtol=1e-14) for x, y in zip(a, b))
    assert np.array_equal(ao.step(p0, g[0], m, v, 1e-2, 4, 0.9, 0.95, 1e-8, 0.1, norm=np.inf, max_norm=2.0)[0], p0)


def test_moments_in_fp32():
    rng = np.random.default_rng(5)
    g, m, v = (rng.standard_normal(300).astype(np.float32) for _ in range(3))
    v = v * v
    for norm, top in ((None, 0.0), (0.5, 1.0), (3.0, 1.0)):
        a, b = ao.moments32(g, m, v, 0.9, 0.95, norm, top)
        assert a.dtype == b.dtype == np.float32
        _, ra, rb = ao.step(np.zeros(300), g, m, v, 0.1, 3, 0.9, 0.95, 1e-8, 0.0, norm, top)
        # a beta, a product and the sum, g's factor: 5 and (squared) 7 roundings of the terms
        assert np.all(np.abs(a - ra) <= 5 * 2.0 ** -24 * (np.abs(0.9 * m) + np.abs(0.1 * g)))
        assert np.all(np.abs(b - rb) <= 7 * 2.0 ** -24 * rb)
    a, b = ao.moments32(np.float32([3.0]), np.float32([1.0]), np.float32([2.0]), 0.5, 0.25)
    assert a[0] == 2.0 and b[0] == 0.5 + 0.75 * 9


def test_state_codes():
    x = np.zeros(300, np.float32)
    x[:5] = [448.0, -1.0, 1e-5, 0.3, -448.0]
    x[130] = 7.0
    codes, s = ao.encode(x)
    assert s.tolist() == [1.0, 7.0 / 448, 1.0] and codes[0] == 0x7E and codes[4] == 0xFE and codes[2] == 0
    assert codes[130] == 0x7E and not codes[256:].any()
    got = ao.decode(codes, s)
    assert got[0] == 448 and got[1] == -1 and abs(got[3] - 0.3) <= 0.3 / 16 and got[130] == np.float32(448) * s[1]
    codes, s = ao.encode(np.abs(x), least=True)
    assert codes[2] == 1 and codes[1] != 0 and codes[5] == 0
