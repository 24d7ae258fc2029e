"""The residual sum between two blocks with the norms on both sides of it, and its gradients, in
float64.  TEST INFRASTRUCTURE ONLY.

u = b, or b / rms(b) w_post; h = r + scale [sigmoid(gate)] u; y = h / rms(h) w of the h that is kept, with
rms(x) = sqrt(mean(x^2) + eps).
"""
from __future__ import annotations

import numpy as np


def _rms(x, eps):
    return np.sqrt((x * x).mean(axis=1, keepdims=True) + eps)


def _sigmoid(z):
    return 1.0 / (1.0 + np.exp(-z))


def _f(x):
    return None if x is None else np.asarray(x, np.float64)


def forward(b, r, gate, w_post, w, eps, scale, keep=lambda h: h):
    """dict(h, kept, y): `keep` rounds h to the type that it is kept in."""
    b, r, gate, w_post, w = map(_f, (b, r, gate, w_post, w))
    h = r
    if b is not None:
        u = b if w_post is None else b / _rms(b, eps) * w_post
        h = r + scale * (u if gate is None else _sigmoid(gate)[:, None] * u)
    kept = keep(h)
    return dict(h=h, kept=kept, y=None if w is None else kept / _rms(kept, eps) * w)


def backward(b, h, gate, w_post, w, dy, dh, eps, scale):
    """dict(dr, db, dgate, dw, dw_post) (None where there is no such input) from the kept h, with the sums of magnitudes
    that each result is made of under "size": what a bound is relative to."""
    b, h, gate, w_post, w, dy, dh = map(_f, (b, h, gate, w_post, w, dy, dh))
    some = next(x for x in (dh, dy, h, b) if x is not None)
    T, D = some.shape
    g = np.zeros((T, D)) if dh is None else dh.copy()
    out, size = dict(db=None, dgate=None, dw=None, dw_post=None), {}
    gs = np.abs(g)
    if w is not None:
        out["dw"], size["dw"] = np.zeros(D), np.zeros(D)
        if dy is not None:
            q = 1.0 / _rms(h, eps)
            e, n = dy * w, h * q
            g += q * (e - n * (e * n).mean(axis=1, keepdims=True))
            gs = gs + q * (np.abs(e) + np.abs(n) * np.abs(e * n).mean(axis=1, keepdims=True))
            out["dw"], size["dw"] = (dy * n).sum(axis=0), np.abs(dy * n).sum(axis=0)
    out["dr"], size["dr"] = g, gs
    f, fs = scale * g, abs(scale) * gs
    if gate is not None:
        s = _sigmoid(gate)[:, None]
        p = 1.0 if w_post is None else w_post / _rms(b, eps)
        f, fs = f * s, fs * s
        out["dgate"] = ((1 - s) * f * (b * p)).sum(axis=1)
        size["dgate"] = ((1 - s) * fs * np.abs(b * p)).sum(axis=1)
    if w_post is not None:
        q = 1.0 / _rms(b, eps)
        n = b * q
        out["dw_post"], size["dw_post"] = (f * n).sum(axis=0), (fs * np.abs(n)).sum(axis=0)
        e, es = f * w_post, fs * np.abs(w_post)
        f = q * (e - n * (e * n).mean(axis=1, keepdims=True))
        fs = q * (es + np.abs(n) * (es * np.abs(n)).mean(axis=1, keepdims=True))
    out["db"], size["db"] = f, fs
    out["size"] = size
    return out
