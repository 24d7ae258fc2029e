"""The residual sum with the norms on both of its sides on the GPU (through the C ABI) against the float64 oracle.

Tolerances, u = 2^-24, half = 2^-8 for bf16 and u for fp32:
* h: without gate and w_post one fused multiply-add, with them 64 bits for a bf16 residual: rounded to fp32 (u), then to
  its type (half), 2^-45 of its terms' sizes for the 64-bit sums' sake; with them and an fp32 residual in fp32: 1 / rms(b)
  15 u as below, scale sigmoid(gate) 8 u, three products and the sum 4 u: 32 u of the sizes;
* y, from the h that the call stored: a sum of squares adds at most 16 values a lane and 6 lane steps in fp32 (22 u,
  positive terms; waves are joined in 64 bits), mean, eps, root and reciprocal 4 u, so q = 1 / rms is off by 15 u
  and y = h q w by 17 u: 24 u, and half;
* dr: q (e - h m), m = sum(e h) / D q^2: 2 u a term, 22 u the sum, 3 * 15 + 4 u for m and q, 3 u the rest: 80 u of the
  sizes that it is made of, and half;
* dw: terms dy (h q) 17 u, summed in 64 bits, rounded to fp32 twice: 24 u of their sizes (past 4096 columns the sums of up to
  16 rows are fp32: 16 u more, also of dw_post);
* db, dgate: g 80 u, scale sigmoid(gate) 8 u, a second sum and its use 80 u, p 15 u thrice: 256 u, and half;
* dw_post: g 80 u, 8 u, b p 17 u, rounded twice: 128 u;
* 2^-126 absolute, where a result may be subnormal (2^-100 for sums of products of such).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mixture_experts_layer_31_amd as moe
from oracle import norm_oracle as no

pytestmark = pytest.mark.gpu
U, TINY = 2.0 ** -24, 2.0 ** -100
F, B = torch.float32, torch.bfloat16
TYPE = {F: moe.MOE_TYPE_F32, B: moe.MOE_TYPE_BF16}
HALF = {F: U, B: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    moe.lib()


def _rows(T, D, pad, off, t, fill):
    buf = torch.full((off + T * (D + pad) + 16,), 55.0, dtype=t, device="cuda")
    v = buf[off:off + T * (D + pad)].view(T, D + pad)[:, :D]
    v.copy_(fill if isinstance(fill, torch.Tensor) else torch.full((T, D), float(fill)))
    return buf, v


def _clean(buf, T, D, pad, off):
    assert (buf[:off] == 55).all() and (buf[off + T * (D + pad):] == 55).all()
    assert (buf[off:off + T * (D + pad)].view(T, D + pad)[:, D:] == 55).all()


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _check(T, D, io=B, res=B, wt=F, block=True, post=False, gated=False, pre=True, dh_in=True, pad=0, off=0, scale=1.0,
           eps=1e-6, in_place=False, seed=0, std=1.0, rows=None):
    print(f"[case] norm T={T} D={D} io={io} res={res} w={wt} block={block} post={post} gate={gated} pre={pre} pad={pad} off={off} "
          f"in_place={in_place}", flush=True)
    g = torch.Generator().manual_seed(seed + T * 31 + D)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    mk = lambda t, fill, o=0: _rows(T, D, pad, (off + o) % 8, t, fill)  # noqa: E731
    bufs = {}

    def put(name, t, fill, o=0):
        bufs[name] = (*mk(t, fill, o), (off + o) % 8)
        return bufs[name][1]

    b = put("b", io, (rows if rows is not None else rnd(T, D)) * std) if block else None
    r = put("r", res, rnd(T, D) * 2 * std, 1)
    w = (1 + 0.1 * rnd(D)).to(wt).cuda() if pre else None
    w_post = (1 + 0.1 * rnd(D)).to(wt).cuda() if post else None
    gate = rnd(T).cuda() if gated else None
    r0 = _np(r)
    h = r if in_place else put("h", res, np.nan, 2)
    y = put("y", io, np.nan, 3) if pre else None
    d = moe.make_norm_desc(T, D, TYPE[io], TYPE[res], TYPE[wt], eps, scale, *[D + pad] * 4)
    assert moe.moe_norm_fwd(d, b, r, gate, w_post, w, h if block or in_place else None, y) == moe.MOE_OK
    torch.cuda.synchronize()
    f = no.forward(_np(b), r0, _np(gate), _np(w_post), _np(w), np.float64(np.float32(eps)), np.float64(np.float32(scale)))
    if block:
        size = np.abs(r0) + np.abs(f["h"] - r0)
        terms = 32 * U if res == F and (post or gated) else 2.0 ** -45
        assert np.all(np.abs(_np(h) - f["h"]) <= (HALF[res] + U) * np.abs(f["h"]) * 1.01 + terms * size + TINY)
    kept = _np(h) if block else r0
    if pre:
        ref = no.forward(None, kept, None, None, _np(w), np.float64(np.float32(eps)), 0.0)["y"]
        assert np.all(np.abs(_np(y) - ref) <= (HALF[io] + 24 * U) * np.abs(ref) + TINY)

    # backward from the stored h
    hk = h if block else r
    dy = put("dy", io, rnd(T, D) * 0.1, 4) if pre else None
    dh = put("dh", res, rnd(T, D) * 0.1, 5) if dh_in else None
    dh0 = _np(dh)
    db = put("db", io, np.nan, 6) if block else None
    dr = dh if in_place and dh_in else put("dr", res, np.nan, 7)
    new = lambda n: torch.full((n,), np.nan, device="cuda")  # noqa: E731
    dgate, dwp, dw = (new(T) if gated else None), (new(D) if post else None), (new(D) if pre else None)
    scratch = torch.full((moe.moe_norm_scratch_bytes(d),), 0xA5, dtype=torch.uint8, device="cuda")
    assert moe.moe_norm_bwd(d, b if post or gated else None, hk if pre else None, gate, w_post, w, dy, dh, db, dr, dgate, dwp, dw,
                            scratch) == moe.MOE_OK
    torch.cuda.synchronize()
    ref = no.backward(_np(b), kept, _np(gate), _np(w_post), _np(w), _np(dy), dh0, np.float64(np.float32(eps)),
                      np.float64(np.float32(scale)))
    got = dict(dr=dr, db=db, dgate=dgate, dw=dw, dw_post=dwp)
    fold = 16 if D > 4096 else 0
    roundings = dict(dr=80, db=256, dgate=256, dw=24 + fold, dw_post=128 + fold)
    half = dict(dr=HALF[res], db=HALF[io], dgate=U, dw=U, dw_post=U)
    for k, v in got.items():
        if v is not None:
            bound = roundings[k] * U * ref["size"][k] * (1 + half[k]) + half[k] * np.abs(ref[k]) + TINY
            err = np.abs(_np(v) - ref[k])
            assert np.all(err <= bound), (k, float((err - bound).max()), float((err / (ref["size"][k] + 1e-300)).max() / U))
    for buf, _, o in bufs.values():
        _clean(buf, T, D, pad, o)


@pytest.mark.parametrize("D", [4, 5, 6, 8, 12, 15, 17, 31, 120, 130, 250, 300, 1300, 2500, 3500, 4097, 6500, 8191, 9001])
def test_rows_that_do_not_fill_their_threads(D):
    """Rows of bf16 whose last loads are moved back to their end, with weights of both types, padding and odd addresses."""
    _check(7, D, wt=B, post=True, gated=True, pad=3, off=1)
    _check(9, D, wt=F, pad=1, off=5)


@pytest.mark.parametrize("D", [1, 2, 3, 7, 8, 9, 63, 64, 65, 100, 511, 512, 513, 1000, 1024, 1025, 2048, 2049, 4096, 4099, 5000, 8192,
                               8193, 16384])
def test_widths(D):
    _check(5, D)
    _check(3, D, io=F, res=F, post=True, gated=True, pad=3, off=1, scale=0.5)
    _check(4, D, io=B, res=F, post=True, pad=1, off=3)
    _check(2, D, io=F, res=B, gated=True, wt=B, off=5, scale=-2.0)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 17, 1023, 1024, 1025, 2500, 5000])
def test_rows(T):
    _check(T, 200, io=B, res=B, post=True, gated=True)
    _check(T, 72, io=B, res=F)


def test_more_rows_than_workgroups_of_the_forward():
    _check(16411, 40, io=F, res=F, post=True)
    _check(4200, 1100)


@pytest.mark.parametrize("io", [F, B])
@pytest.mark.parametrize("res", [F, B])
@pytest.mark.parametrize("wt", [F, B])
def test_parts(io, res, wt):
    """What may be left out, with every type."""
    for block, post, gated, pre in ((True, False, False, True), (True, True, False, True), (True, False, True, True),
                                    (True, True, True, True), (False, False, False, True), (True, False, False, False),
                                    (True, True, True, False), (True, True, False, False), (True, False, True, False)):
        for dh_in in (True, False):
            _check(9, 136, io, res, wt, block, post, gated, pre, dh_in, pad=2, off=1, scale=0.7)


def test_in_place():
    for post in (False, True):
        _check(30, 520, in_place=True, post=post)
        _check(30, 2056, res=F, in_place=True, post=post, pad=5, off=3)
    _check(7, 100, block=False, in_place=True)


def test_rows_of_zeros_and_small_and_large_values():
    z = torch.zeros(4, 300)
    _check(4, 300, io=F, res=F, post=True, rows=z)          # a block that puts out nothing
    _check(4, 300, io=F, res=F, post=True, std=1e-30)       # eps rules
    _check(4, 300, io=F, res=F, post=True, std=1e12, eps=0.0)
    _check(4, 300, io=F, res=F, std=1e-3, eps=1e-12, scale=0.0)


def test_residual_in_bf16_is_the_rounded_sum():
    """With a norm and a gate: every value as 64-bit arithmetic rounds it, to fp32 and then to bf16."""
    T, D = 300, 1000
    g = torch.Generator().manual_seed(5)
    b, r = torch.randn(T, D, generator=g).bfloat16(), torch.randn(T, D, generator=g).bfloat16()
    gate, wp = torch.randn(T, generator=g), 1 + 0.1 * torch.randn(D, generator=g)
    h = torch.zeros(T, D, dtype=B, device="cuda")
    d = moe.make_norm_desc(T, D, scale=0.5)
    assert moe.moe_norm_fwd(d, b.cuda(), r.cuda(), gate.cuda(), wp.cuda(), None, h, None) == moe.MOE_OK
    torch.cuda.synchronize()
    f = no.forward(_np(b), _np(r), _np(gate), _np(wp), None, np.float64(np.float32(1e-6)), 0.5)
    want = torch.from_numpy(f["h"]).float().bfloat16()
    # 300000 values, each off with a chance of 2^-52 over 2^-24 of landing next to a border of fp32's
    assert torch.equal(h.cpu(), want)


def test_values_that_are_not_numbers_stay_in_their_row():
    T, D = 6, 200
    mk = lambda: torch.randn(T, D, device="cuda")  # noqa: E731
    b, r, dy, dh = mk(), mk(), mk(), mk()
    b[1, 3], b[2, 4], r[3, 199] = np.nan, np.inf, np.nan
    w = torch.ones(D, device="cuda")
    d = moe.make_norm_desc(T, D, moe.MOE_TYPE_F32, moe.MOE_TYPE_F32)
    h, y, db, dr = (torch.zeros(T, D, device="cuda") for _ in range(4))
    dw, dwp = torch.zeros(D, device="cuda"), torch.zeros(D, device="cuda")
    scratch = torch.zeros(moe.moe_norm_scratch_bytes(d), dtype=torch.uint8, device="cuda")
    moe.check(moe.moe_norm_fwd(d, b, r, None, w, w, h, y))
    moe.check(moe.moe_norm_bwd(d, b, h, None, w, w, dy, dh, db, dr, None, dwp, dw, scratch))
    torch.cuda.synchronize()
    assert torch.isnan(y[[1, 2, 3]]).any(dim=1).all() and torch.isnan(dw).any()
    for t in (h, y, db, dr):
        assert torch.isfinite(t[[0, 4, 5]]).all()


def test_no_rows():
    e = lambda *s: torch.empty(*s, dtype=B, device="cuda")  # noqa: E731
    d = moe.make_norm_desc(0, 100)
    w, dw, dwp = torch.ones(100, device="cuda"), torch.full((100,), np.nan, device="cuda"), torch.full((100,), np.nan, device="cuda")
    assert moe.moe_norm_fwd(d, e(0, 100), e(0, 100), None, None, w, e(0, 100), e(0, 100)) == moe.MOE_OK
    scratch = torch.zeros(moe.moe_norm_scratch_bytes(d), dtype=torch.uint8, device="cuda")
    assert moe.moe_norm_bwd(d, e(0, 100), e(0, 100), None, w, w, e(0, 100), e(0, 100), e(0, 100), e(0, 100), None, dwp, dw,
                            scratch) == moe.MOE_OK
    torch.cuda.synchronize()
    assert not dw.any() and not dwp.any()


def test_gradient_by_differences():
    """The returned gradient against differences of the float64 forward, in every input."""
    T, D, eps, scale = 2, 6, 1e-2, 1.5
    g = torch.Generator().manual_seed(8)
    v = {k: torch.randn(*s, generator=g) for k, s in dict(b=(T, D), r=(T, D), gate=(T,), w_post=(D,), w=(D,), dy=(T, D),
                                                          dh=(T, D)).items()}
    c = {k: x.cuda() for k, x in v.items()}
    d = moe.make_norm_desc(T, D, moe.MOE_TYPE_F32, moe.MOE_TYPE_F32, eps=eps, scale=scale)
    h, y, db, dr = (torch.zeros(T, D, device="cuda") for _ in range(4))
    dgate, dwp, dw = torch.zeros(T, device="cuda"), torch.zeros(D, device="cuda"), torch.zeros(D, device="cuda")
    scratch = torch.zeros(moe.moe_norm_scratch_bytes(d), dtype=torch.uint8, device="cuda")
    moe.check(moe.moe_norm_fwd(d, c["b"], c["r"], c["gate"], c["w_post"], c["w"], h, y))
    moe.check(moe.moe_norm_bwd(d, c["b"], h, c["gate"], c["w_post"], c["w"], c["dy"], c["dh"], db, dr, dgate, dwp, dw, scratch))
    x = {k: _np(t) for k, t in v.items()}

    def loss(x):
        f = no.forward(x["b"], x["r"], x["gate"], x["w_post"], x["w"], np.float64(np.float32(eps)), scale)
        return (f["y"] * x["dy"]).sum() + (f["h"] * x["dh"]).sum()

    step = 1e-5
    for k, got in (("b", db), ("r", dr), ("gate", dgate), ("w_post", dwp), ("w", dw)):
        got = _np(got)
        for i in np.ndindex(x[k].shape):
            lo, hi = (dict(x, **{k: x[k].copy()}) for _ in range(2))
            lo[k][i] -= step
            hi[k][i] += step
            diff = (loss(hi) - loss(lo)) / (2 * step)
            # step^2 of a third derivative (below 100 here) and fp32's roundings of a sum of sizes below 50
            assert abs(diff - got[i]) <= 1e-8 + 256 * U * 50, (k, i)


def test_same_bits_other_stream_graph_and_two_at_once():
    jobs = []
    for seed in (1, 2):
        torch.manual_seed(seed)
        T, D = 1500, 1030
        mk = lambda: torch.randn(T, D, device="cuda").bfloat16()  # noqa: E731
        w, wp, gate = torch.rand(D, device="cuda"), torch.rand(D, device="cuda"), torch.randn(T, device="cuda")
        d = moe.make_norm_desc(T, D, scale=0.5)
        b, r, dy, dh = mk(), mk(), mk(), mk()
        out = [torch.zeros(T, D, dtype=B, device="cuda") for _ in range(4)] + \
              [torch.zeros(n, device="cuda") for n in (T, D, D)]
        jobs.append((d, b, r, gate, wp, w, dy, dh, out, torch.zeros(moe.moe_norm_scratch_bytes(d), dtype=torch.uint8, device="cuda")))

    def step(j):
        d, b, r, gate, wp, w, dy, dh, (h, y, db, dr, dgate, dwp, dw), scratch = j
        moe.check(moe.moe_norm_fwd(d, b, r, gate, wp, w, h, y))
        moe.check(moe.moe_norm_bwd(d, b, h, gate, wp, w, dy, dh, db, dr, dgate, dwp, dw, scratch))

    refs = []
    for j in jobs:
        step(j)
        torch.cuda.synchronize()
        refs.append([o.clone() for o in j[8]])
    same = lambda k: all(torch.equal(a, o) for a, o in zip(refs[k], jobs[k][8]))  # noqa: E731
    sides = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(20):
        for j, side in zip(jobs, sides):
            with torch.cuda.stream(side):
                step(j)
    torch.cuda.synchronize()
    assert same(0) and same(1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(jobs[0])
    for _ in range(3):
        for o in jobs[0][8]:
            o.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        assert same(0)
        step(jobs[0])
        torch.cuda.synchronize()
        assert same(0)


def test_binding_refuses_what_does_not_fit():
    T, D = 4, 32
    d = moe.make_norm_desc(T, D)
    mk = lambda dt=B, dev="cuda", rows=T, cols=D: torch.zeros(rows, cols, dtype=dt, device=dev)  # noqa: E731
    w = torch.ones(D, device="cuda")
    good = [mk(), mk(), None, None, w, mk(), mk()]
    assert moe.moe_norm_fwd(d, *good) == moe.MOE_OK
    for k, bad in ((0, mk(dev="cpu")), (0, mk(F)), (1, mk(rows=3)), (1, mk(cols=31)), (5, mk(cols=33)), (6, mk(F)), (4, w[:31]),
                   (4, w.bfloat16()), (2, torch.zeros(3, device="cuda")), (3, w.double()), (6, mk().t())):
        args = list(good)
        args[k] = bad
        assert moe.moe_norm_fwd(d, *args) == moe.MOE_EINVAL, k
    scratch = torch.zeros(moe.moe_norm_scratch_bytes(d), dtype=torch.uint8, device="cuda")
    good = [None, mk(), None, None, w, mk(), mk(), mk(), mk(), None, None, torch.zeros(D, device="cuda"), scratch]
    assert moe.moe_norm_bwd(d, *good) == moe.MOE_OK
    for k, bad in ((1, mk(F)), (5, mk(rows=3)), (7, mk(dev="cpu")), (8, mk(cols=33)), (11, torch.zeros(31, device="cuda")),
                   (12, scratch.cpu()), (12, None)):
        args = list(good)
        args[k] = bad
        assert moe.moe_norm_bwd(d, *args) == moe.MOE_EINVAL, k
    args = list(good)
    args[12] = scratch[:-16]
    assert moe.moe_norm_bwd(d, *args) == moe.MOE_ESCRATCH


def test_offsets_past_2_31_elements():
    T, D, ld = 1030, 72, 2 ** 21 + 8
    print(f"[case] norm large T={T} ld={ld}", flush=True)
    bufs = [torch.zeros(T * ld, dtype=B, device="cuda") for _ in range(4)]
    assert bufs[0].numel() > 2 ** 31
    b, r, h, y = (v.view(T, ld)[:, :D] for v in bufs)
    b.copy_(torch.randn(T, D, device="cuda"))
    r.copy_(torch.randn(T, D, device="cuda"))
    w = torch.rand(D, device="cuda") + 0.5
    d = moe.make_norm_desc(T, D, ld_b=ld, ld_r=ld, ld_h=ld, ld_y=ld)
    moe.check(moe.moe_norm_fwd(d, b, r, None, w, w, h, y))
    torch.cuda.synchronize()
    f = no.forward(_np(b), _np(r), None, _np(w), _np(w), np.float64(np.float32(1e-6)), 1.0)
    assert np.all(np.abs(_np(h) - f["h"]) <= (HALF[B] + U) * 1.01 * np.abs(f["h"]) + 2.0 ** -40)
    ref = no.forward(None, _np(h), None, None, _np(w), np.float64(np.float32(1e-6)), 0.0)["y"]
    assert np.all(np.abs(_np(y) - ref) <= (HALF[B] + 24 * U) * np.abs(ref) + TINY)
    # b and r into db and dr, y and h as the upstream gradients
    dw, dwp = torch.zeros(D, device="cuda"), torch.zeros(D, device="cuda")
    scratch = torch.zeros(moe.moe_norm_scratch_bytes(d), dtype=torch.uint8, device="cuda")
    out = [torch.zeros(T * ld, dtype=B, device="cuda") for _ in range(2)]
    db, dr = (v.view(T, ld)[:, :D] for v in out)
    moe.check(moe.moe_norm_bwd(d, b, h, None, w, w, y, h, db, dr, None, dwp, dw, scratch))
    torch.cuda.synchronize()
    ref = no.backward(_np(b), _np(h), None, _np(w), _np(w), _np(y), _np(h), np.float64(np.float32(1e-6)), 1.0)
    for k, v, n, half in (("db", db, 256, HALF[B]), ("dr", dr, 80, HALF[B]), ("dw", dw, 24, U), ("dw_post", dwp, 128, U)):
        assert np.all(np.abs(_np(v) - ref[k]) <= n * U * 1.01 * ref["size"][k] + half * np.abs(ref[k]) + TINY), k
