"""A training step of one block as a user makes it, in a row on one stream: the norm ahead of the layer, the router's
logits as a block-scaled product, the gate with its bias and groups, the layer, the residual sum with a norm on both sides
of it, all their backward passes with the balance loss's gradient, the bias's step, the gradients' norm and AdamW.  Each
result against the float64 oracle of its own step on that step's inputs from the device, with the tolerances of the tests of
the single operators (test_gpu_gate, test_gpu_norm, test_gpu_adamw; the layer's 1e-2 is test_gpu_parity's).  Then steps
captured once and replayed between eager ones.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mixture_experts_layer_31_amd as moe
import moe_inputs as mi
from oracle import adamw_oracle as ao
from oracle import balance_oracle as bo
from oracle import gate_oracle as go
from oracle import moe_oracle as orc
from oracle import norm_oracle as no
from tests.layer_harness import Layer, rel_err

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = moe.MOE_TYPE_BF16, moe.MOE_TYPE_F32
EPS, SCALE, TOP = 1e-6, 0.5, 0.5
BETA = (0.9, 0.95)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    moe.lib()


def _np(t):
    return t.double().cpu().numpy()


def _ld(n):
    return (n + 15) // 16 * 16


class Block:
    def __init__(self, cfg, groups, top_groups, e4m3):
        self.cfg, self.groups, self.top_groups = cfg, groups, top_groups
        T, D, E, K = cfg.T, cfg.D, cfg.E, cfg.K
        self.L = L = Layer(cfg, mi.make_inputs(cfg))
        g = torch.Generator().manual_seed(cfg.seed)
        new = lambda *s, t=torch.float32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
        rnd = lambda *s, by=1.0: (torch.randn(s, generator=g) * by).cuda()  # noqa: E731
        bf, u8 = torch.bfloat16, torch.uint8
        self.r = rnd(T, D).to(bf)
        self.wr = rnd(E, D, by=D ** -0.5).to(bf)
        self.w_in, self.w_post, self.w_out = (1 + rnd(D, by=0.1) for _ in range(3))
        self.gate = rnd(T)
        self.dy, self.dh = rnd(T, D, by=0.1).to(bf), rnd(T, D, by=0.1).to(bf)
        self.bias, self.counts = rnd(E, by=0.05), new(E + 1, t=torch.int32)
        self.z, self.dz, self.mean_p, self.losses = new(T, E), new(T, E), new(E), new(2)
        self.dlosses = torch.tensor([0.0, 1e-3], device="cuda")  # the z-loss; the bias keeps the balance
        self.codes, self.scales = new(E, _ld(D), t=u8), new((E + 127) // 128, (D + 127) // 128)
        self.h, self.y = new(T, D, t=bf), new(T, D, t=bf)
        self.dr, self.dr_in = new(T, D, t=bf), new(T, D, t=bf)
        self.dw_in, self.dw_post, self.dw_out, self.dgate = new(D), new(D), new(D), new(T)
        self.nd = moe.make_norm_desc(T, D, eps=EPS, scale=SCALE)
        self.gd = moe.make_gate_desc(T, E, K, groups=groups, top_groups=top_groups, scale=2.5)
        self.gd_add = moe.make_gate_desc(T, E, K, groups=groups, top_groups=top_groups, scale=2.5,
                                         flags=moe.MOE_GATE_RENORM | moe.MOE_GATE_ACCUMULATE)
        self.mm = moe.make_block_mm_desc(T, E, D, a_type=BF, c_type=F32)
        self.room = new(max(moe.moe_norm_scratch_bytes(self.nd), moe.moe_balance_scratch_bytes(L.desc),
                            moe.moe_block_mm_scratch_bytes(self.mm), moe.moe_grad_scratch_bytes(5)), t=u8)
        self.lr, self.step, self.norm = torch.tensor([1e-2], device="cuda"), new(1, t=torch.int32), new(1)
        self.params = [L.w1.view(-1), L.w2.view(-1), self.w_in, self.w_post, self.w_out]
        self.grads = [L.dw1.view(-1), L.dw2.view(-1), self.dw_in, self.dw_post, self.dw_out]
        self.masters = [p.float() if p.dtype == bf else None for p in self.params]
        self.e4m3, self.decay = e4m3, [0.1, 0.1, 0.0, 0.0, 0.0]
        n = [p.numel() for p in self.params]
        st = lambda: [new(k, t=u8 if e4m3 else torch.float32) for k in n]  # noqa: E731
        sc = lambda: [new((k + 127) // 128) for k in n] if e4m3 else None  # noqa: E731
        self.m, self.v, self.ms, self.vs = st(), st(), sc(), sc()
        self.opt = moe.make_adamw_list(self.params, self.grads, self.m, self.v, self.masters, self.ms, self.vs, self.decay)
        self.ad = moe.make_adamw_desc(*BETA, 1e-8, moe.MOE_TYPE_E4M3 if e4m3 else F32)
        self.list = moe.make_grad_list(self.grads)
        moe.check(moe.moe_block_quant(moe.make_block_quant_desc(E, D, BF, moe.MOE_SCALE_BLOCK), self.wr, self.codes, self.scales))

    def run(self):
        L, ok, room = self.L, moe.check, self.room
        ok(moe.moe_norm_fwd(self.nd, None, self.r, None, None, self.w_in, None, L.x))
        ok(moe.moe_block_mm(self.mm, L.x, None, self.codes, self.scales, self.z, room))
        ok(moe.moe_gate_fwd(self.gd, self.z, self.bias, L.idx, L.w))
        ok(moe.moe_balance_fwd(L.desc, self.z, L.idx, None, self.counts, self.mean_p, self.losses, room))
        L.fwd()
        ok(moe.moe_norm_fwd(self.nd, L.y, self.r, self.gate, self.w_post, self.w_out, self.h, self.y))
        ok(moe.moe_norm_bwd(self.nd, L.y, self.h, self.gate, self.w_post, self.w_out, self.dy, self.dh, L.dy, self.dr,
                            self.dgate, self.dw_post, self.dw_out, room))
        L.bwd()
        ok(moe.moe_balance_bwd(L.desc, self.z, None, self.counts, self.dlosses, None, None, None, self.dz))
        ok(moe.moe_gate_bwd(self.gd_add, self.z, L.idx, L.dprob, self.dz))
        ok(moe.moe_norm_bwd(self.nd, None, self.r, None, None, self.w_in, L.dx, self.dr, None, self.dr_in, None, None,
                            self.dw_in, room))
        ok(moe.moe_gate_bias(self.counts, 1e-3, self.bias))
        ok(moe.moe_grad_norm(self.list, self.norm, room))
        self.step += 1
        ok(moe.moe_adamw(self.ad, self.opt, self.lr, self.step, self.norm, TOP))

    def state(self):
        torch.cuda.synchronize()
        assert self.L.check() == moe.MOE_OK
        L = self.L
        every = [L.x, self.z, L.idx, L.w, self.counts, L.y, self.h, self.y, L.dy, self.dr, self.dgate, L.dx, L.dprob, self.dz,
                 self.dr_in, self.bias, self.norm, self.step, *self.params, *self.grads, *self.m, *self.v]
        return [t.clone() for t in every + [w for w in self.masters if w is not None] + (self.ms or []) + (self.vs or [])]


def _check_norms(S, before):
    L = S.L
    r, h, y = _np(S.r), _np(S.h), _np(S.y)
    w_in, w_post, w_out = (before[k] for k in ("w_in", "w_post", "w_out"))
    eps = np.float64(np.float32(EPS))
    ref = no.forward(None, r, None, None, w_in, eps, 0.0)["y"]
    assert np.all(np.abs(_np(L.x) - ref) <= (2.0 ** -8 + 24 * U) * np.abs(ref))
    f = no.forward(_np(L.y), r, _np(S.gate), w_post, w_out, eps, SCALE)
    assert np.all(np.abs(h - f["h"]) <= (2.0 ** -8 + 2 * U) * np.abs(f["h"]) + 2.0 ** -45 * (np.abs(r) + np.abs(f["h"] - r)))
    ref = no.forward(None, h, None, None, w_out, eps, 0.0)["y"]
    assert np.all(np.abs(y - ref) <= (2.0 ** -8 + 24 * U) * np.abs(ref))
    for got, ref in (
            (dict(dr=S.dr, db=L.dy, dgate=S.dgate, dw=S.dw_out, dw_post=S.dw_post),
             no.backward(_np(L.y), h, _np(S.gate), w_post, w_out, _np(S.dy), _np(S.dh), eps, SCALE)),
            (dict(dr=S.dr_in, dw=S.dw_in), no.backward(None, r, None, None, w_in, _np(L.dx), _np(S.dr), eps, SCALE))):
        for k, v in got.items():
            n = dict(dr=80, db=256, dgate=256, dw=24, dw_post=128)[k]
            half = U if k in ("dgate", "dw", "dw_post") else 2.0 ** -8
            assert np.all(np.abs(_np(v) - ref[k]) <= n * U * 1.01 * ref["size"][k] + half * np.abs(ref[k]) + 2.0 ** -100), k


def _check_gate(S, before):
    cfg, L = S.cfg, S.L
    z = S.z.cpu().numpy()
    f = go.forward(z, before["bias"], cfg.K, "sigmoid", S.groups, S.top_groups, 2, True, 2.5)
    idx = L.idx.cpu().numpy()
    assert np.array_equal(idx, f["idx"])
    assert np.all(np.abs(_np(L.w) - f["w"]) <= 1.01 * U * f["w"])
    counts = S.counts.cpu().numpy()
    assert np.array_equal(counts, np.append(np.bincount(idx.reshape(-1), minlength=cfg.E), cfg.T))
    assert np.array_equal(S.bias.cpu().numpy(), go.bias_step(counts[:cfg.E], 1e-3, before["bias"]))
    # the z-loss's gradient (test_gpu_balance's bound), then the gate's on top of it
    dl = np.float32([0.0, 1e-3]).astype(np.float64)
    b = bo.forward(z, idx)
    zl, dw = bo.backward(z, idx, None, dl, b), _np(L.dprob)
    zk = z.astype(np.float64)
    d = ((zk.max(axis=1, keepdims=True) - zk).max() + cfg.E / 16 + 77) * U
    e = d + 4 * U * (np.abs(b["lse"] - zk.max(axis=1)) + np.abs(b["lse"]))
    c = 2 * dl[1] / cfg.T
    bound = b["p"] * (c * np.abs(b["lse"])[:, None] * (2 * d + 12 * U) + c * e[:, None])
    p = np.take_along_axis(f["s"], idx, 1)
    v = p / p.sum(axis=1, keepdims=True)
    a = np.abs(2.5 * dw)
    each = np.zeros_like(bound)
    np.put_along_axis(each, idx, v * (a + (v * a).sum(axis=1, keepdims=True)), 1)
    ref = zl + go.backward(z, idx, dw, "sigmoid", True, 2.5)
    assert np.all(np.abs(_np(S.dz) - ref) <= bound + 3 * U * each + U * (np.abs(ref) + np.abs(zl)) + 2.0 ** -126)


def _check_layer(S, before):
    L = S.L
    idx, w = L.idx.cpu().numpy(), L.w.cpu().numpy()
    x, dy = (t.float().cpu().numpy() for t in (L.x, L.dy))
    w1, w2 = (before[k].reshape(t.shape).astype(np.float32) for k, t in (("p0", L.w1), ("p1", L.w2)))
    f = orc.forward(x, idx, w, w1, w2)
    b = orc.backward(dy, x, idx, w, w1, w2, f)
    out = L.outputs()
    errs = {k: rel_err(out[k], v) for k, v in (("y", f["y"]), *((k, b[k]) for k in ("dx", "dw1", "dw2", "dprob")))}
    assert all(e <= 1e-2 for e in errs.values()), errs


def _check_step(S, before):
    grads = [_np(t) for t in S.grads]
    full = np.sqrt(sum((g ** 2).sum() for g in grads))
    norm, t, lr = float(S.norm), int(S.step), float(S.lr)
    assert abs(norm - full) <= 2.0 ** -23 * full and norm > TOP
    for k, g in enumerate(grads):
        p0, m0, v0 = (before[f"{x}{k}"] for x in "pmv")
        if S.masters[k] is not None:
            p0 = before[f"w{k}"]
        m32, v32 = ao.moments32(g, m0, v0, *BETA, norm, TOP)
        if S.e4m3:
            (cm, sm), (cv, sv) = ao.encode(m32), ao.encode(np.sqrt(v32), least=True)
            assert all(np.array_equal(a.cpu().numpy(), b) for a, b in ((S.m[k], cm), (S.v[k], cv), (S.ms[k], sm), (S.vs[k], sv)))
        else:
            assert np.array_equal(S.m[k].cpu().numpy(), m32) and np.array_equal(S.v[k].cpu().numpy(), v32)
        p, m, v = ao.step(p0, g, m0, v0, lr, t, *BETA, 1e-8, S.decay[k], norm, TOP)
        terms = BETA[0] * np.abs(m0) + (1 - BETA[0]) * np.abs(g) * TOP / norm
        size = np.abs(p - p0 * (1 - lr * S.decay[k])) + lr / (1 - BETA[0] ** t) * terms / (np.sqrt(v / (1 - BETA[1] ** t)) + 1e-8)
        got = _np(S.params[k] if S.masters[k] is None else S.masters[k])
        assert np.all(np.abs(got - p) <= 2 * U * np.abs(p0) + 20 * U * size + U * np.abs(p))
        if S.masters[k] is not None:
            assert torch.equal(S.params[k], S.masters[k].to(torch.bfloat16))


def _before(S):
    out = {k: _np(getattr(S, k)) for k in ("w_in", "w_post", "w_out")}
    out["bias"] = S.bias.cpu().numpy()
    for k, p in enumerate(S.params):
        out[f"p{k}"] = _np(p)
        if S.masters[k] is not None:
            out[f"w{k}"] = _np(S.masters[k])
        if S.e4m3:
            out[f"m{k}"] = ao.decode(S.m[k].cpu().numpy(), S.ms[k].cpu().numpy())
            root = ao.decode(S.v[k].cpu().numpy(), S.vs[k].cpu().numpy())
            out[f"v{k}"] = root * root
        else:
            out[f"m{k}"], out[f"v{k}"] = _np(S.m[k]), _np(S.v[k])
    return out


@pytest.mark.parametrize("name,groups,top,e4m3", [("small_bf16", 4, 2, False), ("mid_bf16", 1, 1, True), ("dead_bf16", 3, 2, True),
                                                  ("wide_bf16", 2, 1, False)])
def test_steps(name, groups, top, e4m3):
    print(f"[case] block {name} groups={groups}/{top} e4m3={e4m3}", flush=True)
    S = Block(mi.CONFIGS[name], groups, top, e4m3)
    for _ in range(2):
        before = _before(S)
        S.run()
        S.state()
        _check_norms(S, before)
        _check_gate(S, before)
        _check_layer(S, before)
        _check_step(S, before)


def test_captured_steps():
    print("[case] captured block steps", flush=True)
    a, b = (Block(mi.CONFIGS["small_bf16"], 4, 2, True) for _ in range(2))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run()
    for k in range(5):
        a.run()
        want = a.state()
        if k == 2:
            b.run()
        else:
            g.replay()
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(want, b.state())), k
