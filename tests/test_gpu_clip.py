"""Global gradient norm and clipping on the GPU (through the C ABI) against float64.

norm: squares and sums in 64 bits (relative 2^-53 each, far below), one rounding to fp32: 2^-24
relative, doubled for the 64-bit sums' sake.  Clipped values: c = max / norm and the product round
once each, on top of the norm's error: 3 * 2^-24 relative + half a step of the type (2^-8 for bf16)
and of its smallest normal number's step below it.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mixture_experts_layer_31_amd as moe

pytestmark = pytest.mark.gpu
F, B = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    moe.lib()


def _tensors(seed, spec):
    """spec: (n, type, first element in its buffer); values of uneven size per tensor."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for n, t, off in spec:
        x = torch.randn(n, generator=g) * 2.0 ** float(torch.randint(-20, 4, (1,), generator=g))
        buf = torch.full((n + off + 9,), 55.0, dtype=t, device="cuda")
        buf[off:off + n] = x.to(t).cuda()
        out.append((buf, buf[off:off + n]))
    return out


def _norm(lst):
    norm = torch.full((1,), np.nan, device="cuda")
    scratch = torch.full((moe.moe_grad_scratch_bytes(len(lst)),), 0xFF, dtype=torch.uint8, device="cuda")
    assert moe.moe_grad_norm(lst, norm, scratch) == moe.MOE_OK
    return norm


def _ref_norm(xs):
    return float(np.sqrt(sum(float((x.double() ** 2).sum()) for x in xs)))


def _check(spec, name, seed=1, shift=0, share=0.3):
    print(f"[case] clip {name} {len(spec)} tensors, {sum(s[0] for s in spec)} values", flush=True)
    src = _tensors(seed, spec)
    xs = [v for _, v in src]
    ref = _ref_norm(xs)
    old = [v.cpu().double().numpy() for v in xs]
    for in_place in (False, True):
        dst = src if in_place else _tensors(seed + 1, [(n, t, (o + shift) % 9) for n, t, o in spec])
        lst = moe.make_grad_list(xs, [v for _, v in dst])
        norm = _norm(lst)
        torch.cuda.synchronize()
        assert abs(float(norm) - ref) <= 2.0 ** -23 * ref
        top = ref * share if ref else 1.0
        assert moe.moe_grad_clip(lst, norm, top) == moe.MOE_OK
        torch.cuda.synchronize()
        by = np.float64(np.float32(top)) / ref if ref > top else 1.0
        for (buf, v), x, (n, t, o) in zip(dst, old, spec):
            got = v.cpu().double().numpy()
            half = 2.0 ** -8 if t == B else 2.0 ** -24
            assert np.all(np.abs(got - x * by) <= (half + 3 * 2.0 ** -24) * np.abs(x * by) + 2.0 ** -133), name
            off = v.storage_offset()
            assert (buf[:off] == 55).all() and (buf[off + n:] == 55).all()  # the neighbours


@pytest.mark.parametrize("t", [F, B])
def test_lengths_and_alignments(t):
    for off in range(9):
        _check([(n, t, off) for n in (1, 2, 3, 5, 8, 9, 16, 17, 100)], f"short, {off}", shift=off % 3)
    for n in (4096, 8191, 8192, 8193, 16384, 100003):
        _check([(n, t, 0), (n, t, 1)], "chunks", shift=1)


def test_mixed_lists():
    rng = np.random.default_rng(2)
    for count in (1, 7, 95, 96, 97, 200, 300):
        spec = [(int(np.exp(rng.uniform(0, 9))), F if rng.random() < 0.4 else B, int(rng.integers(0, 9)))
                for _ in range(count)]
        spec[count // 2] = (0, F, 0)  # an empty tensor among them
        _check(spec, "mixed", seed=count, shift=int(rng.integers(0, 4)))
    _check([(0, F, 0)], "empty only")


def test_below_the_limit_is_a_copy():
    spec = [(1000, F, 1), (3000, B, 2)]
    _check(spec, "unclipped", share=2.0)
    src = [v for _, v in _tensors(3, spec)]
    dst = [torch.empty_like(v) for v in src]
    lst = moe.make_grad_list(src, dst)
    norm = _norm(lst)
    for top in (float(norm), float(norm) * 2):  # at the limit, and below it
        moe.check(moe.moe_grad_clip(lst, norm, top))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(src, dst))
    moe.check(moe.moe_grad_clip(lst, norm, 0.0))
    torch.cuda.synchronize()
    assert not any(d.any() for d in dst)


def test_values_past_fp32_squares():
    for v in (1e30, 3e38, 1e-30, 1e-44):
        x = torch.full((5000,), v, device="cuda")
        ref = _ref_norm([x])
        n = float(_norm(moe.make_grad_list([x])))
        assert (n == np.inf) if ref > 3.4028236e38 else abs(n - ref) <= 2.0 ** -23 * ref + 2.0 ** -149, v


def test_nan_and_inf():
    for bad in (float("nan"), float("inf")):
        x, y = torch.ones(300, device="cuda"), torch.ones(70, dtype=B, device="cuda")
        x[299] = bad
        out = [torch.zeros_like(x), torch.zeros_like(y)]
        lst = moe.make_grad_list([x, y], out)
        norm = _norm(lst)
        moe.check(moe.moe_grad_clip(lst, norm, 1.0))
        torch.cuda.synchronize()
        if bad != bad:
            assert np.isnan(float(norm)) and all(torch.isnan(o).all() for o in out)
        else:  # 1 / inf = 0 everywhere, inf * 0 at the infinity itself
            assert float(norm) == np.inf and not out[1].any() and not out[0][:299].any() and torch.isnan(out[0][299])


def test_empty_list():
    lst = moe.make_grad_list([])
    assert float(_norm(lst)) == 0.0
    assert moe.moe_grad_clip(lst, torch.zeros(1, device="cuda"), 1.0) == moe.MOE_OK


def test_same_bits_other_stream_and_graph():
    xs = [v for _, v in _tensors(5, [(70001, B, 3), (513, F, 1), (40000, F, 0)])]
    out = [torch.empty_like(v) for v in xs]
    lst = moe.make_grad_list(xs, out)
    norm = torch.zeros(1, device="cuda")
    scratch = torch.empty(moe.moe_grad_scratch_bytes(3), dtype=torch.uint8, device="cuda")

    def step():
        moe.check(moe.moe_grad_norm(lst, norm, scratch))
        moe.check(moe.moe_grad_clip(lst, norm, 0.5))

    step()
    torch.cuda.synchronize()
    ref = [norm.clone()] + [o.clone() for o in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        for o in [norm, *out]:
            o.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, [norm, *out]))
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, [norm, *out]))


def test_binding_refuses_what_is_elsewhere():
    x, norm = torch.ones(10, device="cuda"), torch.ones(1, device="cuda")
    lst, room = moe.make_grad_list([x]), torch.zeros(moe.moe_grad_scratch_bytes(1), dtype=torch.uint8)
    assert moe.moe_grad_norm(lst, norm, room) == moe.MOE_EINVAL  # scratch in host memory
    assert moe.moe_grad_norm(lst, norm.cpu(), room.cuda()) == moe.MOE_EINVAL
    lst.device = 1  # gradients of another GPU than the current one
    assert moe.moe_grad_norm(lst, norm, room.cuda()) == moe.MOE_EINVAL
    assert moe.moe_grad_clip(lst, norm, 1.0) == moe.MOE_EINVAL
    assert moe.moe_grad_clip(moe.make_grad_list([x]), x, 1.0) == moe.MOE_EINVAL  # the norm among the gradients


def test_offsets_past_2_31_elements():
    n = 2 ** 31 + 1003
    print(f"[case] clip large n={n}", flush=True)
    x = torch.full((n,), 0.5, dtype=B, device="cuda")
    x[-5:] = 2.0
    lst = moe.make_grad_list([x])
    norm = _norm(lst)
    ref = np.sqrt((n - 5) * 0.25 + 5 * 4.0)
    moe.check(moe.moe_grad_clip(lst, norm, float(ref) / 4))
    torch.cuda.synchronize()
    assert abs(float(norm) - ref) <= 2.0 ** -23 * ref
    # a quarter of each, within half a step of bf16 and the norm's rounding
    for part, want in ((x[:10], 0.125), (x[2 ** 31 - 8:2 ** 31 + 8], 0.125), (x[-5:], 0.5)):
        assert (part.float() - want).abs().max() <= want * (2.0 ** -8 + 3 * 2.0 ** -24)
    assert bool((x[:-5] == x[0]).all())


def test_two_streams_at_once():
    """Two lists on two streams, each with scratch of its own."""
    jobs = []
    for seed in (1, 2):
        xs = [v for _, v in _tensors(seed, [(300000, B, 3), (513, F, 1), (90000, F, 0)])]
        out = [torch.empty_like(v) for v in xs]
        lst = moe.make_grad_list(xs, out)
        jobs.append((lst, xs, out, torch.zeros(1, device="cuda"),
                     torch.empty(moe.moe_grad_scratch_bytes(3), dtype=torch.uint8, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for lst, _, _, norm, scratch, side in jobs:
            with torch.cuda.stream(side):
                moe.check(moe.moe_grad_norm(lst, norm, scratch))
                moe.check(moe.moe_grad_clip(lst, norm, 0.5))
    torch.cuda.synchronize()
    for lst, xs, out, norm, _, _ in jobs:
        got, n = [o.clone() for o in out], float(norm)
        one = _norm(lst)
        moe.check(moe.moe_grad_clip(lst, one, 0.5))
        torch.cuda.synchronize()
        assert float(one) == n and all(torch.equal(a, b) for a, b in zip(got, out))
