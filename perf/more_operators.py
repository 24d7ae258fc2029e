"""What the rest of a training step around the MoE layer is measured on.

Three kinds of call, beside those of perf/operators.py:

* ``gate``: the router's choice by sigmoid or softmax scores with a balancing
  bias and groups of experts, and the gradient of its weights into the logits;
* ``norm``: the residual sum between two blocks (the block's output with an
  optional norm, gate and scale of its own) and the next block's RMS norm, and
  their backward pass;
* ``adamw``: one optimizer step over a list of tensors, states in fp32 or in
  e4m3 with a scale for each 128.

``run`` computes them in elementary torch operations where ``own`` is false and
through the package's entry points where it is true.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0


def listed():
    return [
        # one token of a decoding step: latency
        dict(name="gate-token", op="gate", T=1, E=128, K=8, groups=1, top=1, best=2, score="sigmoid",
             io="f32", bias=True, renorm=True, scale=1.0, pad=0, train=False),
        # one sequence of 16384 tokens over 128 experts, top-8, a bias in place of a balance loss
        dict(name="gate-128", op="gate", T=16384, E=128, K=8, groups=1, top=1, best=2, score="sigmoid",
             io="f32", bias=True, renorm=True, scale=1.0, pad=0, train=True),
        # softmax scores as they are, an odd number of tokens, groups that are no power of two, padded bf16 rows
        dict(name="gate-odd", op="gate", T=4099, E=160, K=6, groups=8, top=3, best=1, score="softmax",
             io="bf16", bias=False, renorm=False, scale=16.0, pad=5, train=True),
        # a long batch over 256 experts in eight groups, of which four may be chosen from
        dict(name="gate-groups", op="gate", T=65536, E=256, K=8, groups=8, top=4, best=2, score="sigmoid",
             io="f32", bias=True, renorm=True, scale=2.5, pad=0, train=True),
        # one token of a decoding step through a block's end and the next norm
        dict(name="norm-token", op="norm", T=1, D=2048, io="bf16", res="bf16", post=False, gate=False, pad=0, train=False),
        # the layer's rows, one sequence, residual in bf16
        dict(name="norm-layer", op="norm", T=16384, D=2048, io="bf16", res="bf16", post=False, gate=False, pad=0, train=True),
        # fp32 and odd: a small model's width that is no multiple of anything, rows with padding
        dict(name="norm-odd", op="norm", T=1363, D=1001, io="f32", res="f32", post=True, gate=False, pad=3, train=True),
        # a norm on both sides of a gated block, a wider model, residual in fp32
        dict(name="norm-gated", op="norm", T=16384, D=4096, io="bf16", res="f32", post=True, gate=True, pad=0, train=True),
        # a small model's tensors in fp32: latency
        dict(name="adamw-small", op="adamw", count=6, total=200000, share=1.0, master=False, states="f32"),
        # weights of an expert-parallel rank's layer in bf16 with masters, its router's in fp32
        dict(name="adamw-layer", op="adamw", layer=True, E=16, D=2048, F=768, master=True, states="f32"),
        # a whole layer's, where memory is short: states in e4m3, no masters
        dict(name="adamw-e4m3", op="adamw", layer=True, E=128, D=2048, F=768, master=False, states="e4m3"),
        # odd, unaligned tensors of both types, as views into flat buffers
        dict(name="adamw-many", op="adamw", count=60, total=40000000, share=0.3, master=False, states="e4m3"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["gate", "norm", "adamw"])
    if op == "gate":
        groups = rng.choice([1, 1, 2, 3, 4, 8, 16])
        each = _log(rng, 2 if groups > 1 else 8, 256 // groups)
        top = rng.randint(1, groups)
        K = rng.randint(1, min(8, top * each))
        # one expert's renormalised weight is 1 and has no gradient
        return dict(op=op, T=_log(rng, 1, 65536), E=groups * each, K=K, groups=groups, top=top, best=rng.choice([1, 2]),
                    score=rng.choice(["sigmoid", "softmax"]), io=rng.choice(["f32", "bf16"]),
                    bias=rng.random() < 0.7, renorm=K > 1 and rng.random() < 0.7, scale=rng.choice([1.0, 2.5]),
                    pad=rng.choice([0, 0, 3]), train=rng.random() < 0.8)
    if op == "norm":
        D = _log(rng, 8, 8192)
        return dict(op=op, T=_log(rng, 1, min(65536, 16384 * 4096 // D)), D=D, io=rng.choice(["bf16", "bf16", "f32"]),
                    res=rng.choice(["bf16", "f32"]), post=rng.random() < 0.5, gate=rng.random() < 0.5,
                    pad=rng.choice([0, 0, 5]), train=rng.random() < 0.8)
    return dict(op=op, count=_log(rng, 1, 60), total=_log(rng, 1000, 100000000), share=rng.choice([0.0, 0.3, 1.0]),
                master=rng.random() < 0.5, states=rng.choice(["f32", "e4m3"]))


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _type(io):
    return torch.bfloat16 if io == "bf16" else torch.float32


def _rows(T, D, pad, t, g=None, std=1.0):
    """[T, D] with pad more elements between its rows."""
    x = torch.zeros(T, D + pad, dtype=t, device=DEV)
    if g is not None:
        x[:, :D] = torch.randn(T, D, generator=g, device=DEV) * std
    return x[:, :D]


def _prepare_gate(c, g):
    T, E, K, t = c["T"], c["E"], c["K"], _type(c["io"])
    popular = torch.randn(E, generator=g, device=DEV) * 0.7  # popular and unpopular experts
    z = _rows(T, E, c["pad"], t, g)
    z += popular.to(t)
    s = dict(z=z, bias=None, idx=torch.empty(T, K, dtype=torch.int32, device=DEV), w=torch.empty(T, K, device=DEV))
    if c["bias"]:  # what some thousand steps have moved it by
        s["bias"] = torch.randn(E, generator=g, device=DEV) * (0.1 if c["score"] == "sigmoid" else 0.5 / E)
    if c["train"]:
        s["dw"] = torch.randn(T, K, generator=g, device=DEV) * 1e-3
        s["dz"] = _rows(T, E, c["pad"], t)
    return s


def _prepare_norm(c, g):
    T, D, io, res, pad = c["T"], c["D"], _type(c["io"]), _type(c["res"]), c["pad"]
    s = dict(b=_rows(T, D, pad, io, g), r=_rows(T, D, pad, res, g, 2.0), h=_rows(T, D, pad, res), y=_rows(T, D, pad, io),
             w=1.0 + 0.1 * torch.randn(D, generator=g, device=DEV), gate=None, w_post=None, eps=1e-6, scale=1.0)
    if c["post"]:
        s["w_post"] = 1.0 + 0.1 * torch.randn(D, generator=g, device=DEV)
    if c["gate"]:
        s["gate"], s["scale"] = torch.randn(T, generator=g, device=DEV), 0.5
    if c["train"]:
        s.update(dy=_rows(T, D, pad, io, g, 1e-2), dh=_rows(T, D, pad, res, g, 1e-2), db=_rows(T, D, pad, io),
                 dr=_rows(T, D, pad, res), dw=torch.empty(D, device=DEV),
                 dgate=torch.empty(T, device=DEV) if c["gate"] else None,
                 dw_post=torch.empty(D, device=DEV) if c["post"] else None,
                 scratch=torch.empty(8 * 1024 * (D + 64), dtype=torch.uint8, device=DEV))
    return s


def _tensors(c):
    """(length, fp32?, elements left free before it, weight decay) of each tensor of the list."""
    if c.get("layer"):  # [E, 2F, D] and [E, D, F] in bf16, the router's [E, D] and a norm's [D] in fp32
        E, D, F = c["E"], c["D"], c["F"]
        return [(E * 2 * F * D, False, 0, 0.1), (E * D * F, False, 0, 0.1), (E * D, True, 0, 0.1), (D, True, 0, 0.0)]
    # a few large ones and many small, odd ones
    rng = np.random.default_rng([c["count"], c["total"]])
    part = np.exp(rng.normal(0.0, 1.5, c["count"]))
    return [(max(1, int(c["total"] * p)), bool(rng.random() < c["share"]), int(rng.integers(0, 8)),
             0.1 if rng.random() < 0.7 else 0.0) for p in part / part.sum()]


def _prepare_adamw(c, g):
    """The flat buffers that a trainer keeps, and each tensor's part of them."""
    spec, e4m3 = _tensors(c), c["states"] == "e4m3"
    size = dict(f32=0, bf16=0, state=0, scale=0)
    parts = []
    for n, single, first, decay in spec:
        t = "f32" if single else "bf16"
        parts.append((t, size[t] + first, size["state"], size["scale"], n, decay))
        size[t] += first + n
        size["state"] += -(-n // 128) * 128
        size["scale"] += -(-n // 128)
    flat = {}
    for t in ("f32", "bf16"):
        flat["p_" + t] = torch.empty(size[t], dtype=_type(t), device=DEV).normal_(0.0, 0.02, generator=g)
        flat["g_" + t] = torch.empty(size[t], dtype=_type(t), device=DEV).normal_(0.0, 1e-3, generator=g)
    if c["master"]:
        # what the bf16 parameters were rounded from
        flat["master"] = flat["p_bf16"].float() * (1.0 + 1e-3 * torch.rand(size["bf16"], generator=g, device=DEV))
        flat["p_bf16"].copy_(flat["master"])
    # states of a run under way: |m| about 3e-4, v about 1e-6, uneven
    n = size["state"]
    m = torch.empty(n, device=DEV).normal_(0.0, 3e-4, generator=g)
    v = torch.empty(n, device=DEV).normal_(0.0, 1.0, generator=g).exp_().mul_(1e-3)
    if e4m3:
        flat["m"], flat["m_scale"] = _coded(m.view(-1, 128))
        flat["v"], flat["v_scale"] = _coded(v.view(-1, 128), least=True)
    else:
        flat["m"], flat["v"] = m, v.square_()
    tensors = []
    for t, at, st, sc, n, decay in parts:
        e = dict(param=flat["p_" + t][at:at + n], grad=flat["g_" + t][at:at + n], m=flat["m"][st:st + n], v=flat["v"][st:st + n],
                 master=None, m_scale=None, v_scale=None, decay=decay)
        if c["master"] and t == "bf16":
            e["master"] = flat["master"][at:at + n]
        if e4m3:
            runs = -(-n // 128)
            e.update(m_scale=flat["m_scale"][sc:sc + runs], v_scale=flat["v_scale"][sc:sc + runs])
        tensors.append(e)
    s = dict(flat=flat, tensors=tensors, lr=torch.tensor([3e-4], device=DEV), step=torch.tensor([1000], dtype=torch.int32, device=DEV),
             norm=torch.tensor([1.7], device=DEV), max_norm=1.0, beta1=0.9, beta2=0.95, eps=1e-8)
    if own:  # the list of buffers that a trainer keeps
        import mixture_experts_layer_31_amd as moe
        s["list"] = moe.make_adamw_list(
            [e["param"] for e in tensors], [e["grad"] for e in tensors], [e["m"] for e in tensors], [e["v"] for e in tensors],
            masters=[e["master"] for e in tensors] if c["master"] else None,
            m_scales=[e["m_scale"] for e in tensors] if e4m3 else None,
            v_scales=[e["v_scale"] for e in tensors] if e4m3 else None, weight_decay=[e["decay"] for e in tensors])
        s["desc"] = moe.make_adamw_desc(0.9, 0.95, 1e-8, moe.MOE_TYPE_E4M3 if e4m3 else moe.MOE_TYPE_F32)
    return s


def prepare(case, seed):
    g = _gen(seed)
    s = dict(gate=_prepare_gate, norm=_prepare_norm, adamw=_prepare_adamw)[case["op"]](case, g)
    s["case"] = case
    return s


# ---------------------------------------------------------------- the plain forms

def _scores(z, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + (-z).exp())
    e = (z - z.amax(dim=1, keepdim=True)).exp()
    return e / e.sum(dim=1, keepdim=True)


def _largest(c, k):
    """Places of the k largest of the last axis, descending, ties to the lower one."""
    return torch.argsort(c, dim=-1, descending=True, stable=True)[..., :k]


def _gate(s):
    c, z = s["case"], s["z"]
    T, E, G = c["T"], c["E"], c["groups"]
    # scores next to each other decide which expert is taken: in 64 bits, the choice rounded once
    score = _scores(z.double(), c["score"])
    choice = (score if s["bias"] is None else score + s["bias"].double()).float()
    choice = torch.where(torch.isnan(choice) | (z == -math.inf), -torch.finfo(torch.float32).max, choice)
    if c["top"] < G:
        groups = choice.view(T, G, E // G)
        best = torch.gather(groups, 2, _largest(groups, min(c["best"], E // G)))
        taken = _largest(best.sum(dim=2), c["top"])
        keep = torch.zeros(T, G, dtype=torch.bool, device=DEV).scatter_(1, taken, True)
        choice = torch.where(keep[:, :, None], groups, -math.inf).view(T, E)
    idx = _largest(choice, c["K"])
    w = torch.gather(score, 1, idx)
    if c["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    out = dict(idx=idx.to(torch.int32), w=(w * c["scale"]).float())
    if c["train"]:
        p = _scores(z.float(), c["score"])
        picked, a = torch.gather(p, 1, idx), s["dw"] * c["scale"]
        if c["renorm"]:
            total = picked.sum(dim=1, keepdim=True)
            a = torch.where(total > 0, (a - (picked / total * a).sum(dim=1, keepdim=True)) / total, 0.0)
        if c["score"] == "sigmoid":
            dz = torch.zeros(T, E, device=DEV).scatter_(1, idx, picked * (1.0 - picked) * a)
        else:
            part = torch.zeros(T, E, device=DEV).scatter_(1, idx, a)
            dz = p * (part - (picked * a).sum(dim=1, keepdim=True))
        out["dlogits"] = dz.to(z.dtype)
    return out


def _norm(s):
    c, D = s["case"], s["case"]["D"]
    b, io = s["b"].float(), s["b"].dtype
    by, rb, u = s["scale"], 1.0, s["b"].double()
    # the residual in 64 bits: kept in 16, a value next to a border goes one way or the other
    if s["gate"] is not None:
        by = s["scale"] / (1.0 + (-s["gate"].double()).exp())[:, None]
    if s["w_post"] is not None:
        rb = 1.0 / (u.square().mean(dim=1, keepdim=True) + s["eps"]).sqrt()
        u = u * rb * s["w_post"].double()
        rb = rb.float()
    h = (s["r"].double() + by * u).float().to(s["r"].dtype)
    if s["gate"] is not None:
        by, u = by.float(), u.float()
    x = h.float()  # the residual as it is kept
    rs = 1.0 / (x.square().mean(dim=1, keepdim=True) + s["eps"]).sqrt()
    out = dict(h=h, y=(x * rs * s["w"]).to(io))
    if not c["train"]:
        return out
    dy = s["dy"].float()
    n = x * rs
    e = dy * s["w"]
    dh = s["dh"].float() + rs * (e - n * (e * n).mean(dim=1, keepdim=True))
    out.update(dr=dh.to(h.dtype), dw=(dy * n).sum(dim=0, dtype=torch.float64).float())
    f = by * dh
    if s["gate"] is not None:
        out["dgate"] = (f * u).sum(dim=1) / (1.0 + s["gate"].exp())
    if s["w_post"] is not None:
        nb = b * rb
        out["dw_post"] = (f * nb).sum(dim=0, dtype=torch.float64).float()
        f = f * s["w_post"]
        f = rb * (f - nb * (f * nb).mean(dim=1, keepdim=True))
    out["db"] = f.to(io)
    return out


def _coded(x, least=False):
    """e4m3 values of the rows of x [runs, 128] and their scales; least: what is positive keeps a
    positive code. The divisions are in 64 bits and rounded to 32: a quotient next to the border of
    two codes decides between them."""
    amax = x.abs().amax(dim=1)
    s = torch.where(amax == 0, 1.0, (amax.double() / E4M3_MAX).float())
    q = (x.double() / s.double()[:, None]).float().clamp(-E4M3_MAX, E4M3_MAX)
    if least:
        q = torch.where(x > 0, q.clamp_min(2.0 ** -9), q)
    return q.to(torch.float8_e4m3fn).reshape(-1), s


def _runs(x):
    return torch.nn.functional.pad(x, (0, -x.shape[0] % 128)).view(-1, 128)


def _adamw(s):
    c, e4m3 = s["case"], s["case"]["states"] == "e4m3"
    t = s["step"].double()
    b1, b2, eps, lr = s["beta1"], s["beta2"], s["eps"], s["lr"]
    c1, c2 = (1.0 - b1 ** t).float(), (1.0 - b2 ** t).float()
    by = torch.where(s["norm"] <= s["max_norm"], 1.0, s["max_norm"] / s["norm"])
    for e in s["tensors"]:
        n = e["param"].shape[0]
        g = e["grad"].float() * by
        m, v = e["m"].float(), e["v"].float()
        if e4m3:
            m = (_runs(m) * e["m_scale"][:, None]).view(-1)[:n]
            v = (_runs(v) * e["v_scale"][:, None]).view(-1)[:n].square()
        m = b1 * m + (1.0 - b1) * g
        v = b2 * v + (1.0 - b2) * g.square()
        p = (e["param"] if e["master"] is None else e["master"]).float()
        p = p * (1.0 - lr * e["decay"]) - lr * (m / c1) / ((v / c2).sqrt() + eps)
        e["param"].copy_(p)
        if e["master"] is not None:
            e["master"].copy_(p)
        if e4m3:
            q, scale = _coded(_runs(m))
            e["m"].view(torch.uint8).copy_(q[:n].view(torch.uint8))
            e["m_scale"].copy_(scale)
            q, scale = _coded(_runs(v.sqrt()), least=True)
            e["v"].view(torch.uint8).copy_(q[:n].view(torch.uint8))
            e["v_scale"].copy_(scale)
        else:
            e["m"].copy_(m)
            e["v"].copy_(v)
    return _updated(s)


def _updated(s):
    return {k: v for k, v in s["flat"].items() if not k.startswith("g_") and v.numel()}


# ---------------------------------------------------------------- the package's calls

def _own_gate(s):
    import mixture_experts_layer_31_amd as moe
    c = s["case"]
    d = moe.make_gate_desc(
        c["T"], c["E"], c["K"], score=moe.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else moe.MOE_SCORE_SOFTMAX,
        groups=c["groups"], top_groups=c["top"], group_best=c["best"],
        in_type=moe.MOE_TYPE_BF16 if c["io"] == "bf16" else moe.MOE_TYPE_F32, scale=c["scale"],
        flags=moe.MOE_GATE_RENORM if c["renorm"] else 0, ld_logits=c["E"] + c["pad"], ld_dlogits=c["E"] + c["pad"])
    moe.check(moe.moe_gate_fwd(d, s["z"], s["bias"], s["idx"], s["w"]))
    out = dict(idx=s["idx"], w=s["w"])
    if c["train"]:
        moe.check(moe.moe_gate_bwd(d, s["z"], s["idx"], s["dw"], s["dz"]))
        out["dlogits"] = s["dz"]
    return out


def _own_norm(s):
    import mixture_experts_layer_31_amd as moe
    c, ld = s["case"], s["case"]["D"] + s["case"]["pad"]
    types = dict(bf16=moe.MOE_TYPE_BF16, f32=moe.MOE_TYPE_F32)
    d = moe.make_norm_desc(c["T"], c["D"], io_type=types[c["io"]], res_type=types[c["res"]], eps=s["eps"], scale=s["scale"],
                           ld_b=ld, ld_r=ld, ld_h=ld, ld_y=ld)
    moe.check(moe.moe_norm_fwd(d, s["b"], s["r"], s["gate"], s["w_post"], s["w"], s["h"], s["y"]))
    out = dict(h=s["h"], y=s["y"])
    if c["train"]:
        moe.check(moe.moe_norm_bwd(d, s["b"], s["h"], s["gate"], s["w_post"], s["w"], s["dy"], s["dh"], s["db"], s["dr"],
                                   s["dgate"], s["dw_post"], s["dw"], s["scratch"]))
        out.update(dr=s["dr"], db=s["db"], dw=s["dw"])
        if c["gate"]:
            out["dgate"] = s["dgate"]
        if c["post"]:
            out["dw_post"] = s["dw_post"]
    return out


def _own_adamw(s):
    import mixture_experts_layer_31_amd as moe
    moe.check(moe.moe_adamw(s["desc"], s["list"], s["lr"], s["step"], s["norm"], s["max_norm"]))
    return _updated(s)


def run(state):
    op = state["case"]["op"]
    if own:
        return (_own_gate if op == "gate" else _own_norm if op == "norm" else _own_adamw)(state)
    return (_gate if op == "gate" else _norm if op == "norm" else _adamw)(state)


# ---------------------------------------------------------------- work and the definitions in 64 bits

def work(case):
    if case["op"] == "gate":
        T, E, K, size = case["T"], case["E"], case["K"], 2 if case["io"] == "bf16" else 4
        n = T * E * size + T * K * 8 + (E * 4 if case["bias"] else 0)
        if case["train"]:
            n += T * K * 4 + T * E * size
        return {"bytes": n, "flops": 20 * T * E}
    if case["op"] == "norm":
        T, D = case["T"], case["D"]
        io, res = (2 if case[k] == "bf16" else 4 for k in ("io", "res"))
        n = T * D * (2 * io + 2 * res)
        if case["train"]:
            n *= 2
        return {"bytes": n + D * 16, "flops": T * D * (40 if case["train"] else 10)}
    n = 0
    for length, single, _, _ in _tensors(case):
        # gradient in, parameter in and out (from the master where there is one), states in and out
        param = 8 if single else 10 if case["master"] else 4
        states = 4 + 16 / 128 if case["states"] == "e4m3" else 16
        n += length * ((4 if single else 2) + param + states)
    return {"bytes": n, "flops": 16 * sum(t[0] for t in _tensors(case))}


def _exact_gate(s):
    c = s["case"]
    E, G, K = c["E"], c["groups"], c["K"]
    z = s["z"].double()
    logp = z - torch.logsumexp(z, dim=1, keepdim=True) if c["score"] == "softmax" else torch.nn.functional.logsigmoid(z)
    choice = logp.exp()
    if s["bias"] is not None:
        choice = choice + s["bias"].double()
    # the choice on the host: a stable sort of whole rows by (group is in, choice)
    choice = choice.float().cpu().numpy()
    order = np.argsort(-choice, axis=1, kind="stable")
    if c["top"] < G:
        member = np.sort(choice.reshape(-1, G, E // G), axis=2)[:, :, ::-1]
        score = member[:, :, 0].copy()
        if c["best"] == 2 and E // G > 1:
            score += member[:, :, 1]
        rank = np.argsort(np.argsort(-score, axis=1, kind="stable"), axis=1, kind="stable")
        out = np.take_along_axis(rank, order // (E // G), axis=1) >= c["top"]
        order = np.take_along_axis(order, np.argsort(out, axis=1, kind="stable"), axis=1)
    idx = torch.from_numpy(np.ascontiguousarray(order[:, :K])).to(DEV)
    x = z.clone().requires_grad_()
    p = torch.softmax(x, dim=1) if c["score"] == "softmax" else torch.sigmoid(x)
    w = torch.gather(p, 1, idx)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    w = w * c["scale"]
    out = dict(idx=idx.to(torch.int32), w=w.detach())
    if c["train"]:
        (out["dlogits"],) = torch.autograd.grad((w * s["dw"].double()).sum(), x)
    return out


def _exact_norm(s):
    # the two norms as they are defined, their derivatives by differentiation; the residual is
    # rounded to the type it is kept in before the second norm, whose gradient passes the rounding
    c, D = s["case"], s["case"]["D"]
    leaf = {k: s[k].double().requires_grad_() for k in ("b", "r", "w", "gate", "w_post") if s[k] is not None}
    u = leaf["b"]
    if c["post"]:
        u = u / ((u * u).sum(dim=1, keepdim=True) / D + s["eps"]) ** 0.5 * leaf["w_post"]
    if c["gate"]:
        u = u * torch.sigmoid(leaf["gate"])[:, None]
    h = leaf["r"] + s["scale"] * u
    kept = h + (h.detach().to(s["r"].dtype).double() - h.detach())
    y = kept / ((kept * kept).sum(dim=1, keepdim=True) / D + s["eps"]) ** 0.5 * leaf["w"]
    out = dict(h=h.detach(), y=y.detach())
    if c["train"]:
        total = (y * s["dy"].double()).sum() + (kept * s["dh"].double()).sum()
        grads = dict(zip(leaf, torch.autograd.grad(total, list(leaf.values()))))
        out.update({"d" + k: v for k, v in grads.items()})
    return out


def _exact_code(x, least):
    """Values of the codes and the scales of x in runs of 128: x a number of 32 bits, the scale and the
    quotient rounded to 32 bits by the format's definition, a code the nearest multiple of its
    binade's step, ties to even."""
    n = x.numel()
    t = _runs(x.float().double())
    amax = t.abs().amax(dim=1, keepdim=True)
    s = torch.where(amax == 0, 1.0, amax / E4M3_MAX).float().double()
    v = (t / s).float().double()
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    q = (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
    if least:
        q = torch.where((t > 0) & (q == 0), 2.0 ** -9, q)
    return q.reshape(-1)[:n], s[:, 0]


def _exact_adamw(s):
    e4m3 = s["case"]["states"] == "e4m3"
    out = {k: v.double() for k, v in _updated(s).items()}
    t, b1, b2, lr = int(s["step"]), s["beta1"], s["beta2"], float(s["lr"])
    by = min(1.0, s["max_norm"] / float(s["norm"]))
    for e in s["tensors"]:
        g = e["grad"].double() * by
        m, v = e["m"].double(), e["v"].double()
        if e4m3:
            runs = torch.arange(m.numel(), device=DEV) // 128
            m, v = m * e["m_scale"].double()[runs], (v * e["v_scale"].double()[runs]) ** 2
        m = m + (1.0 - b1) * (g - m)
        v = v + (1.0 - b2) * (g * g - v)
        old = (e["param"] if e["master"] is None else e["master"]).double()
        new = old - lr * (e["decay"] * old + (m / (1.0 - b1 ** t)) / ((v / (1.0 - b2 ** t)) ** 0.5 + s["eps"]))

        def put(name, part, value):  # into the flat buffer at the part's place
            at = part.storage_offset()
            out[name][at:at + part.numel()] = value

        put("p_f32" if e["param"].dtype == torch.float32 else "p_bf16", e["param"], new)
        if e["master"] is not None:
            put("master", e["master"], new)
        if e4m3:
            for name, x in (("m", m), ("v", v.float().double().sqrt())):
                q, scale = _exact_code(x, name == "v")
                put(name, e[name], q)
                put(name + "_scale", e[name + "_scale"], scale)
        else:
            put("m", e["m"], m)
            put("v", e["v"], v)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return (_exact_gate if op == "gate" else _exact_norm if op == "norm" else _exact_adamw)(s)
