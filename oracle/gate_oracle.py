"""The gate's choice, weights and gradient, in float64.  TEST INFRASTRUCTURE ONLY.

s = sigmoid(z) or softmax(z) (0 for a row of only -inf), c = fl32(s + bias), -FLT_MAX where z is -inf or
c is NaN or -inf.  With fewer top groups than groups a group scores the fp32 sum of its best one or two c, and
only the best groups' experts can be chosen.  The K largest c, ties to the lower place; w = scale s, or scale s /
sum s.  Where that sum comes to the end of 64-bit numbers the quotients are those of exp(z - max) over the chosen (of
either score: down there a sigmoid is exp z); 0 where all of those are -inf, or sigmoid scores that are 0 in 64 bits.
"""
from __future__ import annotations

import numpy as np

FLT_MAX = np.finfo(np.float32).max


def scores(z, score):
    z = np.asarray(z, np.float64)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if score == "sigmoid":
            return np.where(z < -600, np.exp(np.minimum(z, 0)), 1.0 / (1.0 + np.exp(-z)))
        m = z.max(axis=1, keepdims=True)
        e = np.where(m == -np.inf, 0.0, np.exp(z - np.where(m == -np.inf, 0.0, m)))
        total = e.sum(axis=1, keepdims=True)
        return np.where(total == 0, 0.0, e / np.where(total == 0, 1.0, total))


def _largest(c, k):
    return np.argsort(-c, axis=-1, kind="stable")[..., :k]


def shares(p, x, score):
    """p / sum p of each row, p the scores of the logits x (p = 0, x = -inf: a slot that takes no part)."""
    total = p.sum(axis=1, keepdims=True)
    m = x.max(axis=1, keepdims=True)
    far = (total < 1e-280) & (m > -np.inf) & ((total > 0) | (score == "softmax"))
    with np.errstate(invalid="ignore", over="ignore"):
        p = np.where(far, np.exp(x - np.where(m == -np.inf, 0.0, m)), p)
    total = p.sum(axis=1, keepdims=True)
    return np.where(total == 0, 0.0, p / np.where(total == 0, 1.0, total)), far


def forward(z, bias, K, score="sigmoid", groups=1, top_groups=1, group_best=2, renorm=True, scale=1.0):
    """dict(idx [T, K], w [T, K], s [T, E], c [T, E])."""
    z = np.asarray(z)
    T, E = z.shape
    s = scores(z, score)
    with np.errstate(invalid="ignore"):
        c = (s if bias is None else s + np.asarray(bias, np.float64)).astype(np.float32)
        c = np.where(np.isnan(c) | (np.asarray(z) == -np.inf), -FLT_MAX, np.maximum(c, -FLT_MAX)).astype(np.float32)
    rank = c.astype(np.float64)
    if top_groups < groups:
        each = E // groups
        best = -np.sort(-c.reshape(T, groups, each), axis=2)[:, :, :min(group_best, each)]
        with np.errstate(over="ignore"):
            total = best[:, :, 0] if best.shape[2] == 1 else best[:, :, 0] + best[:, :, 1]  # in fp32
        taken = np.zeros((T, groups), bool)
        np.put_along_axis(taken, _largest(total, top_groups), True, axis=1)
        rank = np.where(np.repeat(taken, each, axis=1), rank, -np.inf)  # behind every -FLT_MAX
    idx = _largest(rank, K).astype(np.int32)
    w = np.take_along_axis(s, idx, axis=1)
    if renorm:
        w, _ = shares(w, np.take_along_axis(np.asarray(z, np.float64), idx, axis=1), score)
    return dict(idx=idx, w=w * scale, s=s, c=c)


def backward(z, idx, dw, score="sigmoid", renorm=True, scale=1.0):
    """dL/dz [T, E] with idx fixed, by the chain rule through the renormalisation and the score (through the shares themselves
    where the scores' sum comes to the end of 64-bit numbers)."""
    z, idx = np.asarray(z, np.float64), np.asarray(idx)
    T, E = z.shape
    s = scores(z, score)
    ok = (idx >= 0) & (idx < E)
    at = np.where(ok, idx, 0)
    p = np.where(ok, np.take_along_axis(s, at, axis=1), 0.0)
    a = np.where(ok, np.asarray(dw, np.float64) * scale, 0.0)
    t, k = np.nonzero(ok)
    far, dfar = np.zeros((T, 1), bool), np.zeros((T, E))
    if renorm:
        v, far = shares(p, np.where(ok, np.take_along_axis(z, at, axis=1), -np.inf), score)
        # dL/dz of the chosen where a sigmoid's 1 - s is 1
        np.add.at(dfar, (t, idx[t, k]), (v * (a - (v * a).sum(axis=1, keepdims=True)))[t, k])
        total = p.sum(axis=1, keepdims=True)
        safe = np.where((total == 0) | far, 1.0, total)
        a = np.where(total == 0, 0.0, (a - (p / safe * a).sum(axis=1, keepdims=True)) / safe)
    ds = np.zeros((T, E))
    np.add.at(ds, (t, idx[t, k]), a[t, k])
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            dz = s * (1.0 / (1.0 + np.exp(z))) * ds
    else:
        dz = s * (ds - (s * ds).sum(axis=1, keepdims=True))
    return np.where(far, dfar, dz)


def bias_step(counts, step, bias):
    """bias + step where a count is below the mean of all, - step where it is above (in fp32)."""
    counts = [int(c) for c in counts]
    total, E = sum(counts), len(counts)
    sign = np.array([(c * E < total) - (c * E > total) for c in counts], np.float32)
    return np.asarray(bias, np.float32) + sign * np.float32(step)
