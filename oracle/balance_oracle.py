"""Load-balancing loss, z-loss and per-expert counts of the router, in float64.  TEST INFRASTRUCTURE ONLY.

With V the kept tokens, n = |V|, p = softmax(z), f_e the share of V's (token, slot) pairs that
went to expert e and P_e the mean of p_te over V:
    loss0 = E sum_e f_e P_e,    loss1 = mean over V of logsumexp(z_t)^2.
"""
from __future__ import annotations

import numpy as np


def _softmax(z):
    m = z.max(axis=1, keepdims=True)
    e = np.exp(z - m)
    s = e.sum(axis=1, keepdims=True)
    return e / s, (m + np.log(s))[:, 0]


def forward(z, idx, valid=None):
    """dict(counts [E+1], mean_p [E], losses [2], p [n, E], lse [n], keep): idx [T, K], ids outside
    [0, E) not counted."""
    z, idx = np.asarray(z, np.float64), np.asarray(idx)
    T, E = z.shape
    K = idx.shape[1]
    keep = np.arange(T) if valid is None else np.flatnonzero(np.asarray(valid))
    n = len(keep)
    ids = idx[keep].reshape(-1)
    counts = np.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
    if n == 0:
        p, lse = np.zeros((0, E)), np.zeros(0)
        mean_p, losses = np.zeros(E), np.zeros(2)
    else:
        p, lse = _softmax(z[keep])
        mean_p = p.mean(axis=0)
        losses = np.array([E * (counts / (n * K) * mean_p).sum(), (lse ** 2).mean()])
    return dict(counts=np.append(counts, n), mean_p=mean_p, losses=losses, p=p, lse=lse, keep=keep)


def backward(z, idx, valid, dlosses, fwd=None):
    """d (dlosses . losses) / d z, [T, E]."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    K = np.asarray(idx).shape[1]
    f = forward(z, idx, valid) if fwd is None else fwd
    dz = np.zeros((T, E))
    n = len(f["keep"])
    if n:
        share = f["counts"][:E] / (n * K)
        p = f["p"]
        dz[f["keep"]] = p * (dlosses[0] * E / n * (share - (p * share).sum(axis=1, keepdims=True))
                             + dlosses[1] * 2 / n * f["lse"][:, None])
    return dz


def router_part(idx, w, dw, E):
    """The gradient of the renormalised routing weights, w_j (dw_j - sum_k w_k dw_k) at the selected
    experts, [T, E]."""
    idx, w, dw = np.asarray(idx), np.asarray(w, np.float64), np.asarray(dw, np.float64)
    g = w * (dw - (w * dw).sum(axis=1, keepdims=True))
    dz = np.zeros((idx.shape[0], E))
    t, k = np.nonzero((idx >= 0) & (idx < E))
    np.add.at(dz, (t, idx[t, k]), g[t, k])
    return dz
