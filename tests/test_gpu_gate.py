"""The gate on the GPU (through the C ABI) against the float64 oracle.

The choice is compared for equality: it goes by 64-bit scores rounded once to fp32 on both sides.
Tolerances, u = 2^-24, half = 2^-8 for bf16 and u for fp32:
* weights: 64 bits, rounded once to fp32: u relative (2^-40 for the 64-bit sums' sake); of softmax scores that are not
  renormalised the sum of all exps is fp32: with d_i = z_i - z_max, whose rounding and product with log2 e shift an exp
  by 2.5 u |d_i|, on average over the row's probabilities at most 2.5 u ln E (their entropy) <= 18 u, the exp's 2 u, a
  sum by halves 11 u, the reciprocal 2 u and the last rounding: 40 u;
* gradients of sigmoid scores and of renormalised ones: each slot's in 64 bits, rounded to
  fp32, two slots' of one expert added: 3 u of their sizes, and half a step of the type;
* softmax as it is, in fp32: a probability is off by d = (R + E / 16 + 77) u relative, R the largest
  max z - z (z - max rounds by R u, expf 4 u, at most E / 16 + 70 additions, 3 u the rest), s (a - sum s a) so by
  s (|a| + sum s |a|) (2 d + (K + 8) u);
* 2^-126 absolute, where a result may be subnormal;
* the oracle's own: with renormalised softmax scores s_j (0 - sum_k s_k ds_k) is 0 of an expert that is not chosen, and the
  oracle forms that sum of at most 64 terms in 64 bits: it is off by some 16 roundings of 2^-53 of the terms'
  sizes, so by less than 2^-48 s_j sum_k |s_k ds_k|.
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


def _rows(a, t, pad, off=0):
    """On the GPU with `pad` more elements between rows, `off` elements into its buffer."""
    T, E = a.shape
    buf = torch.full((off + T * (E + pad) + 8,), 55.0, dtype=t, device="cuda")
    v = buf[off:off + T * (E + pad)].view(T, E + pad)[:, :E]
    v.copy_(torch.from_numpy(np.ascontiguousarray(a, np.float32)))
    return buf, v


def _check(z, bias, K, score="sigmoid", groups=1, top=1, best=2, renorm=True, scale=1.0, t=F, pad=0, off=0, seed=0,
           add=False, idx=None, name=""):
    T, E = z.shape
    print(f"[case] gate {name} T={T} E={E} K={K} {score} groups={groups}/{top}/{best} renorm={renorm} {t} pad={pad}", flush=True)
    io = moe.MOE_TYPE_F32 if t == F else moe.MOE_TYPE_BF16
    flags = (moe.MOE_GATE_RENORM if renorm else 0) | (moe.MOE_GATE_ACCUMULATE if add else 0)
    d = moe.make_gate_desc(T, E, K, SCORE[score], groups, top, best, io, flags, scale, E + pad, E + pad)
    zbuf, zt = _rows(z, t, pad, off)
    z = zt.float().cpu().numpy()  # as the type holds them
    it = torch.full((T, K), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, K), np.nan, device="cuda")
    bt = None if bias is None else torch.from_numpy(np.float32(bias)).cuda()
    assert moe.moe_gate_fwd(d, zt, bt, it, w) == moe.MOE_OK
    torch.cuda.synchronize()
    f = go.forward(z, None if bias is None else np.float32(bias), K, score, groups, top, best, renorm, scale)
    assert np.array_equal(it.cpu().numpy(), f["idx"]), name
    got = w.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(f["w"]))
    ok = ~np.isnan(got)
    rel = 40 * U if score == "softmax" and not renorm else U + 2.0 ** -40
    assert np.all(np.abs(got - f["w"])[ok] <= (rel * np.abs(f["w"]) + TINY)[ok]), name

    rng = np.random.default_rng(seed)
    dw = rng.standard_normal((T, K)).astype(np.float32)
    if idx is not None:
        it.copy_(torch.from_numpy(idx))
    ids = it.cpu().numpy()
    old = rng.standard_normal((T, E)).astype(np.float32) if add else np.full((T, E), np.nan, np.float32)
    obuf, dz = _rows(old, t, pad, (off + 1) % 8)
    dwt = torch.from_numpy(dw).cuda()
    assert moe.moe_gate_bwd(d, zt, it, dwt, dz) == moe.MOE_OK
    torch.cuda.synchronize()
    ref = go.backward(z, ids, dw, score, renorm, scale)
    ok = (ids >= 0) & (ids < E)
    at = np.where(ok, ids, 0)
    a = np.abs(np.where(ok, dw.astype(np.float64) * scale, 0.0))
    p = np.where(ok, np.take_along_axis(f["s"], at, 1), 0.0)
    each = np.zeros((T, E))
    if renorm:
        total = p.sum(axis=1, keepdims=True)
        v = np.where(total == 0, 0.0, p / np.where(total == 0, 1.0, total))
        size = v * (a + (v * a).sum(axis=1, keepdims=True))
    else:
        size = p * a
    tt, kk = np.nonzero(ok)
    np.add.at(each, (tt, ids[tt, kk]), size[tt, kk])
    bound = 3 * U * each + 2.0 ** -48 * f["s"] * size.sum(axis=1, keepdims=True)
    if score == "softmax" and not renorm:
        R = np.where(np.isfinite(z), z.max(axis=1, keepdims=True) - z, 0).max() if np.isfinite(z).any() else 0
        dd = (R + E / 16 + 77) * U
        aj = np.zeros((T, E))
        np.add.at(aj, (tt, ids[tt, kk]), a[tt, kk])
        bound = f["s"] * (aj + (p * a).sum(axis=1, keepdims=True)) * (2 * dd + (K + 8) * U)
    half = U if t == F else 2.0 ** -8
    if add:
        ref = ref + old
        bound = bound + U * np.abs(ref)
    bound = bound * (1 + half) + half * np.abs(ref) + TINY
    err = np.abs(dz.float().cpu().numpy() - ref)
    assert np.all(err <= bound), (name, float((err - bound).max()))
    # what lies between the rows
    if pad:
        for buf, o in ((zbuf, off), (obuf, (off + 1) % 8)):
            assert (buf[o:o + T * (E + pad)].view(T, E + pad)[:, E:] == 55).all()
            assert (buf[:o] == 55).all() and (buf[o + T * (E + pad):] == 55).all()
    return it, w, dz


def _logits(seed, T, E, spread=1.5):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal((T, E)) * spread).astype(np.float32), rng.standard_normal(E) * 0.1


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 8, 2), (1, 128, 8), (3, 5, 5), (64, 8, 2), (65, 64, 3), (257, 65, 4),
                                   (700, 100, 6), (333, 128, 8), (129, 256, 16), (50, 257, 2), (77, 256, 17), (200, 512, 64),
                                   (41, 513, 3), (37, 1000, 7), (66, 1024, 64)])
def test_shapes(T, E, K, score):
    z, bias = _logits(T * 7 + E, T, E)
    _check(z, bias, K, score, name="bias")
    _check(z, None, K, score, renorm=False, scale=2.5, pad=3, off=1, name="plain")
    _check(z, bias / E, K, score, t=B, pad=1, off=3, name="bf16")


@pytest.mark.parametrize("E,G,top,K", [(16, 2, 1, 8), (16, 8, 3, 4), (160, 8, 3, 6), (256, 8, 4, 8), (96, 3, 2, 7), (100, 5, 2, 9),
                                       (33, 11, 4, 12), (17, 17, 9, 9), (64, 64, 40, 33), (512, 16, 5, 20), (1024, 64, 32, 64),
                                       (990, 33, 7, 30), (1020, 3, 2, 5), (904, 8, 2, 16), (420, 7, 7, 10), (128, 16, 15, 8)])
def test_groups(E, G, top, K):
    for score, best, renorm, t in (("sigmoid", 2, True, F), ("softmax", 1, False, B), ("sigmoid", 1, False, B), ("softmax", 2, True, F)):
        z, bias = _logits(E + G, 61, E)
        _check(z, bias if score == "sigmoid" else bias / E, K, score, G, top, best, renorm, 2.5, t, pad=E % 3, name="groups")


def test_ties_go_to_the_lower_place():
    rng = np.random.default_rng(1)
    z = rng.integers(0, 3, (200, 96)).astype(np.float32)
    for score in SCORE:
        _check(z, None, 8, score, name="ties")
        _check(z, None, 8, score, 8, 3, name="ties in groups")
        _check(np.zeros((5, 96), np.float32), None, 9, score, 4, 2, name="all equal")
    # saturated scores are equal in fp32
    _check(np.float32([[20.0, 30.0, 40.0, 25.0] * 4] * 3), None, 5, name="saturated")


def test_neighbours_of_a_border():
    """Scores an fp32 exp would order otherwise: logits one step of fp32 apart, their scores a step or less."""
    rng = np.random.default_rng(2)
    z = np.tile(rng.standard_normal((400, 1)).astype(np.float32), (1, 64))
    step = rng.integers(-6, 7, z.shape, dtype=np.int32)
    z = (z.view(np.int32) + step).view(np.float32)
    bias = np.zeros(64, np.float32)
    for score in SCORE:
        _check(z, bias, 8, score, name="neighbours")
        _check(z, bias, 8, score, 8, 4, name="neighbours in groups")


def test_masked_experts():
    z, bias = _logits(3, 90, 64)
    rng = np.random.default_rng(3)
    z[rng.random(z.shape) < 0.9] = -np.inf
    z[7] = -np.inf  # nothing is left
    z[8] = -np.inf
    z[8, 5] = 1.0
    for score in SCORE:
        for renorm in (True, False):
            _check(z, bias, 8, score, renorm=renorm, name="masked")
            _check(z, bias, 8, score, 8, 4, renorm=renorm, t=B, name="masked in groups")
    # by the bias
    bias[rng.random(64) < 0.5] = -np.inf
    _check(z, bias, 8, name="masked by the bias")
    # the type's lowest value
    low = np.where(np.isinf(z), np.finfo(np.float32).min, z)
    for score in SCORE:
        _check(low, None, 8, score, name="lowest")


def test_nan_and_inf():
    z, _ = _logits(4, 6, 32)
    z[0, 3], z[1, :], z[2, 4], z[3, 5:] = np.nan, np.nan, np.inf, np.nan
    for score in SCORE:
        for G in (1, 4):
            d = moe.make_gate_desc(6, 32, 4, SCORE[score], G, 2 if G > 1 else 1)
            zt, it, w = torch.from_numpy(z).cuda(), torch.zeros(6, 4, dtype=torch.int32, device="cuda"), torch.zeros(6, 4, device="cuda")
            assert moe.moe_gate_fwd(d, zt, None, it, w) == moe.MOE_OK
            dz = torch.zeros(6, 32, device="cuda")
            assert moe.moe_gate_bwd(d, zt, it, w, dz) == moe.MOE_OK
            torch.cuda.synchronize()
            ids = it.cpu().numpy()
            assert ((ids >= 0) & (ids < 32)).all() and all(len(set(r)) == 4 for r in ids)
            if score == "sigmoid":  # a NaN is chosen last, +inf scores 1
                assert 3 not in ids[0] and ids[2, 0] == 4 and not torch.isnan(w[[0, 2, 4, 5]]).any()
            else:  # the whole row's scores
                assert torch.isnan(w[[0, 1, 2]]).all()
            assert not torch.isnan(w[[4, 5]]).any() and not torch.isnan(dz[[4, 5]]).any()


def test_extreme_logits():
    z, bias = _logits(5, 100, 128, spread=40.0)
    for score in SCORE:
        for renorm in (True, False):
            _check(z, bias, 8, score, renorm=renorm, name="wide")
    _check(np.float32(z * 1e36), None, 8, name="huge")


def test_peaked_softmax():
    """Scores without a bias, chosen by the logits: far apart, below fp32's normal numbers, and equal again as 0."""
    for spread in (0.01, 1.0, 6.0, 25.0, 120.0):
        for t in (F, B):
            z, _ = _logits(11, 300, 96, spread=spread)
            for renorm in (True, False):
                _check(z, None, 8, "softmax", renorm=renorm, t=t, name=f"spread {spread}")
                _check(z, None, 8, "softmax", 8, 3, 1, renorm=renorm, t=t, name=f"spread {spread} in groups")
                _check(z, None, 8, "softmax", 8, 3, 2, renorm=renorm, t=t, name=f"spread {spread} in groups by two")


@pytest.mark.parametrize("E,G,top,K", [(96, 8, 3, 8), (256, 1, 1, 8), (130, 1, 1, 5), (512, 8, 4, 8), (40, 4, 2, 20)])
def test_a_token_alone_and_among_others(E, G, top, K):
    """A token's ids and weights are the same bits whatever stands beside it: rows that are chosen again in 64 bits
    (masked, equal, past the numbers) among others that are not."""
    z, bias = _logits(12, 60, E)
    z[::7, ::3] = -np.inf
    z[5::14] = 0.25
    z[2, 1], z[11, 2], z[23, :] = np.inf, np.nan, -np.inf
    zt = torch.from_numpy(z).cuda()
    bt = torch.from_numpy(np.float32(bias)).cuda()
    for score in SCORE:
        for flags in (0, moe.MOE_GATE_RENORM):
            for b in (None, bt):
                outs = []
                for rows in [range(0, 60), *[range(t, t + 1) for t in range(60)]]:
                    n = len(rows)
                    d = moe.make_gate_desc(n, E, K, SCORE[score], G, top, 2, moe.MOE_TYPE_F32, flags, 2.5)
                    it = torch.full((n, K), -7, dtype=torch.int32, device="cuda")
                    w = torch.full((n, K), 7.0, device="cuda")
                    assert moe.moe_gate_fwd(d, zt[rows.start:rows.stop], b, it, w) == moe.MOE_OK
                    outs.append((it, w))
                alone = [torch.cat(v) for v in zip(*outs[1:])]
                for got, want in zip(alone, outs[0]):
                    assert torch.equal(got.view(torch.int32), want.view(torch.int32)), (score, flags, b is None)


def test_ids_twice_and_out_of_range():
    z, bias = _logits(6, 40, 48)
    rng = np.random.default_rng(6)
    idx = rng.integers(-1, 50, (40, 6)).astype(np.int32)
    idx[:, 1] = idx[:, 0]
    idx[3] = -1
    for score in SCORE:
        for renorm in (True, False):
            _check(z, None, 6, score, renorm=renorm, idx=idx, name="twice")


def test_adds_to_a_gradient():
    z, bias = _logits(7, 130, 100)
    for score in SCORE:
        for renorm in (True, False):
            _check(z, bias, 6, score, renorm=renorm, add=True, pad=2, name="add")


def test_several_workgroups():
    z, bias = _logits(8, 20011, 24)
    _check(z, bias, 3, groups=3, top=2, name="many tokens")
    z, bias = _logits(9, 3001, 300)
    _check(z, bias / 300, 8, "softmax", renorm=False, name="many tokens")


def test_no_tokens():
    d = moe.make_gate_desc(0, 64, 4)
    e = lambda *s, t=F: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    assert moe.moe_gate_fwd(d, e(0, 64), None, e(0, 4, t=torch.int32), e(0, 4)) == moe.MOE_OK
    assert moe.moe_gate_bwd(d, e(0, 64), e(0, 4, t=torch.int32), e(0, 4), e(0, 64)) == moe.MOE_OK


def test_gradient_by_differences():
    z, bias = _logits(10, 3, 12)
    dw = np.random.default_rng(10).standard_normal((3, 4)).astype(np.float32)
    for score in SCORE:
        for renorm in (True, False):
            d = moe.make_gate_desc(3, 12, 4, SCORE[score], flags=moe.MOE_GATE_RENORM if renorm else 0)
            dz, it, w = torch.zeros(3, 12, device="cuda"), torch.zeros(3, 4, dtype=torch.int32, device="cuda"), torch.zeros(3, 4, device="cuda")
            zt = torch.from_numpy(z).cuda()
            moe.check(moe.moe_gate_fwd(d, zt, None, it, w))
            moe.check(moe.moe_gate_bwd(d, zt, it, torch.from_numpy(dw).cuda(), dz))
            idx, got, step = it.cpu().numpy(), dz.cpu().numpy(), 1e-6

            def loss(x):
                s = go.scores(x, score)
                p = np.take_along_axis(s, idx, 1)
                return ((p / p.sum(axis=1, keepdims=True) if renorm else p) * dw).sum()

            for i in np.ndindex(3, 12):
                lo, hi = z.astype(np.float64), z.astype(np.float64)
                lo[i] -= step
                hi[i] += step
                # the difference's own error: step^2 and 2^-52 of the loss (below 8) over the step
                assert abs((loss(hi) - loss(lo)) / (2 * step) - got[i]) <= 2e-8 + 2e-6 * abs(got[i])


@pytest.mark.parametrize("E", [1, 8, 100, 1024, 5000])
def test_bias(E):
    rng = np.random.default_rng(E)
    counts = rng.integers(0, 5, E + 1).astype(np.int32)
    counts[:E // 2] *= 400000000
    bias = rng.standard_normal(E).astype(np.float32)
    ct, bt = torch.from_numpy(counts).cuda(), torch.from_numpy(bias).cuda()
    assert moe.moe_gate_bias(ct, 0.125, bt) == moe.MOE_OK
    torch.cuda.synchronize()
    assert np.array_equal(bt.cpu().numpy(), go.bias_step(counts[:E], 0.125, bias))


def test_same_bits_other_stream_graph_and_two_at_once():
    jobs = []
    for seed in (1, 2):
        z, bias = _logits(seed, 3000, 160)
        d = moe.make_gate_desc(3000, 160, 6, groups=8, top_groups=3, scale=2.5)
        e = lambda *s, t=F: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
        jobs.append((d, torch.from_numpy(z).cuda(), torch.from_numpy(np.float32(bias)).cuda(), e(3000, 6, t=torch.int32),
                     e(3000, 6), torch.randn(3000, 6, device="cuda"), e(3000, 160)))

    def step(j):
        d, z, b, it, w, dw, dz = j
        moe.check(moe.moe_gate_fwd(d, z, b, it, w))
        moe.check(moe.moe_gate_bwd(d, z, it, dw, dz))

    refs = []
    for j in jobs:
        step(j)
        torch.cuda.synchronize()
        refs.append([j[k].clone() for k in (3, 4, 6)])
    sides = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(20):
        for j, side in zip(jobs, sides):
            with torch.cuda.stream(side):
                step(j)
    torch.cuda.synchronize()
    assert all(torch.equal(a, j[k]) for j, r in zip(jobs, refs) for a, k in zip(r, (3, 4, 6)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(jobs[0])
    for _ in range(3):
        for k in (3, 4, 6):
            jobs[0][k].fill_(9)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, jobs[0][k]) for a, k in zip(refs[0], (3, 4, 6)))
        step(jobs[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, jobs[0][k]) for a, k in zip(refs[0], (3, 4, 6)))


def test_binding_refuses_what_does_not_fit():
    d = moe.make_gate_desc(8, 16, 2)
    e = lambda *s, t=F, dev="cuda": torch.zeros(*s, dtype=t, device=dev)  # noqa: E731
    z, it, w, dz, bias = e(8, 16), e(8, 2, t=torch.int32), e(8, 2), e(8, 16), e(16)
    assert moe.moe_gate_fwd(d, z, bias, it, w) == moe.MOE_OK
    for bad in ((z.cpu(), bias, it, w), (z.double(), bias, it, w), (z[:7], bias, it, w), (e(8, 32)[:, ::2], bias, it, w),
                (z.t(), bias, it, w), (z, bias[:15], it, w), (z, bias.double(), it, w), (z, bias, it.long(), w),
                (z, bias, it[:, :1], w), (z, bias, it, w.half()), (z, bias, it, w.cpu()), (e(8, 17)[:, :16], bias, it, w)):
        assert moe.moe_gate_fwd(d, *bad) == moe.MOE_EINVAL
    assert moe.moe_gate_bwd(d, z, it, w, dz) == moe.MOE_OK
    for bad in ((z, it, w, dz.cpu()), (z, it, w, dz.bfloat16()), (z, it, w, dz[:7]), (z, it, w, z), (z, it, w.double(), dz)):
        assert moe.moe_gate_bwd(d, *bad) == moe.MOE_EINVAL
    assert moe.moe_gate_bias(it, 0.1, bias) == moe.MOE_OK  # 16 counts
    for bad in ((it[:7], bias), (it.float(), bias), (it, bias.cpu()), (it, None)):
        assert moe.moe_gate_bias(bad[0], 0.1, bad[1]) == moe.MOE_EINVAL


def test_offsets_past_2_31_elements():
    """The last of 2^31 logits and more, in rows that lie far apart."""
    T, E = 2 ** 20 + 3, 8
    ld = 2048 + 8
    print(f"[case] gate large T={T} ld={ld}", flush=True)
    buf = torch.zeros(T * ld, dtype=B, device="cuda")
    assert buf.numel() > 2 ** 31
    z = buf.view(T, ld)[:, :E]
    z.copy_(torch.randn(T, E, device="cuda"))
    out = torch.full((T * ld,), 7.0, dtype=B, device="cuda")
    dz = out.view(T, ld)[:, :E]
    d = moe.make_gate_desc(T, E, 2, in_type=moe.MOE_TYPE_BF16, ld_logits=ld, ld_dlogits=ld)
    it, w = torch.zeros(T, 2, dtype=torch.int32, device="cuda"), torch.zeros(T, 2, device="cuda")
    moe.check(moe.moe_gate_fwd(d, z, None, it, w))
    dw = torch.randn(T, 2, device="cuda")
    moe.check(moe.moe_gate_bwd(d, z, it, dw, dz))
    torch.cuda.synchronize()
    rows = [0, 1, 2 ** 20 - 1, T - 2, T - 1]
    zs = z[rows].float().cpu().numpy()
    f = go.forward(zs, None, 2)
    assert np.array_equal(it[rows].cpu().numpy(), f["idx"]) and np.allclose(w[rows].cpu().numpy(), f["w"], rtol=2 * U)
    ref = go.backward(zs, f["idx"], dw[rows].cpu().numpy())
    assert np.all(np.abs(dz[rows].float().cpu().numpy() - ref) <= (2.0 ** -8 + 4 * U) * np.abs(ref) + 2.0 ** -40)
    assert bool((out.view(T, ld)[::5000, E:] == 7).all())
