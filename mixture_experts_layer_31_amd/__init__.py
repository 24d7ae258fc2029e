"""Python binding of the MI355X MoE layer's C ABI (include/moe.h).

Argument marshalling only: every step of the layer runs in the HIP library
libmoe_mi355x.so built in-tree by ``mixture_experts_layer_31_amd.build``.  The
functions below carry the C names; tensors are torch tensors on the GPU (or
None for optional pointers) and `stream` defaults to torch's current stream.
Loading fails loudly when the library has not been built: there is no fallback.
The calls of the operators beside the layer (moe_balance_*, moe_block_*, moe_grad_*)
also look at their tensors: one of another type, device or stride than the call takes,
or with too few elements, is MOE_EINVAL.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_mi355x.so")

MOE_FP32, MOE_FP32_BF16GEMM, MOE_BF16, MOE_FP8_BWD, MOE_MXFP8, MOE_FP8 = range(6)
MOE_OK, MOE_EINVAL, MOE_ESCRATCH, MOE_EALIGN, MOE_EUNSUPPORTED, MOE_EHIP, MOE_EINDEX, \
    MOE_ETIMEOUT = 0, -1, -2, -3, -4, -5, -6, -7
MOE_FLAG_OVERLAP = 0x1
MOE_FLAG_QUEUE_TIMEOUT_TEST = 0x2
MOE_FLAG_RECOMPUTE = 0x4
MOE_FLAG_OVERLAP_BWD = 0x8
MOE_FLAG_SERIAL_BWD = 0x10
MOE_NOALLOC_SCRATCH_BYTES = 256 << 20
(MOE_VIEW_XPERM, MOE_VIEW_H, MOE_VIEW_A, MOE_VIEW_O, MOE_VIEW_DYPERM, MOE_VIEW_DH,
 MOE_VIEW_DXPERM, MOE_VIEW_WPERM, MOE_VIEW_Q_ROWS, MOE_VIEW_Q_ROWS_SCALE, MOE_VIEW_Q_TOK_A,
 MOE_VIEW_Q_TOK_A_SCALE, MOE_VIEW_Q_TOK_B, MOE_VIEW_Q_TOK_B_SCALE, MOE_VIEW_QUEUE) = range(15)

MOE_TYPE_F32, MOE_TYPE_BF16, MOE_TYPE_E4M3 = range(3)
MOE_SCALE_TILE, MOE_SCALE_BLOCK = range(2)
MOE_MM_ACCUMULATE = 0x1

# Exported symbols, in the order include/moe.h declares them.
EXPORTS = (
    "moe_scratch_bytes", "moe_wprep_bytes", "moe_prepare_weights", "moe_route",
    "moe_routing_view", "moe_scratch_view", "moe_fwd", "moe_bwd", "moe_fwd_noalloc", "moe_router_fwd",
    "moe_router_bwd", "moe_balance_scratch_bytes", "moe_balance_fwd", "moe_balance_bwd", "moe_block_quant",
    "moe_block_mm_scratch_bytes", "moe_block_mm", "moe_grad_scratch_bytes", "moe_grad_norm", "moe_grad_clip",
    "moe_check", "moe_strerror", "moe_abi_version", "moe_profile_enable", "moe_profile_collect",
    "moe_profile_get", "moe_profile_reset",
)


class moe_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "D", "F", "E", "K", "mode", "flags")]


class moe_block_quant_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "cols", "in_type", "scale")] + \
               [(n, ctypes.c_int64) for n in ("ld_in", "ld_codes", "ld_codes_t")]


class moe_block_mm_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("M", "N", "K", "a_type", "b_scale", "c_type", "flags")] + \
               [(n, ctypes.c_int64) for n in ("lda", "ldb", "ldc")]


class moe_grad(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("type", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class MoeError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {strerror(code)} ({code})")


_lib = None
_vp, _sz, _i32, _i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64
_dp = ctypes.POINTER(moe_desc)


def lib() -> ctypes.CDLL:
    """The loaded HIP library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run `python -m mixture_experts_layer_31_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        sig = {
            "moe_scratch_bytes": (_sz, [_dp]),
            "moe_wprep_bytes": (_sz, [_dp]),
            "moe_prepare_weights": (_i32, [_dp, _vp, _vp, _vp, _sz, _vp]),
            "moe_route": (_i32, [_dp, _vp, _vp, _sz, _vp]),
            "moe_routing_view": (_i32, [_dp, _vp, _sz] + [ctypes.POINTER(_vp)] * 4),
            "moe_scratch_view": (_i32, [_dp, _vp, _sz, _i32, ctypes.POINTER(_vp), ctypes.POINTER(_sz)]),
            "moe_fwd": (_i32, [_dp] + [_vp] * 8 + [_sz, _vp]),
            "moe_bwd": (_i32, [_dp] + [_vp] * 10 + [_sz, _vp]),
            "moe_fwd_noalloc": (_i32, [_dp] + [_vp] * 8),
            "moe_router_fwd": (_i32, [_dp, _vp, _vp, _vp, _vp]),
            "moe_router_bwd": (_i32, [_dp, _vp, _vp, _vp, _vp, _vp]),
            "moe_balance_scratch_bytes": (_sz, [_dp]),
            "moe_balance_fwd": (_i32, [_dp] + [_vp] * 7 + [_sz, _vp]),
            "moe_balance_bwd": (_i32, [_dp] + [_vp] * 9),
            "moe_block_quant": (_i32, [ctypes.POINTER(moe_block_quant_desc)] + [_vp] * 6),
            "moe_block_mm_scratch_bytes": (_sz, [ctypes.POINTER(moe_block_mm_desc)]),
            "moe_block_mm": (_i32, [ctypes.POINTER(moe_block_mm_desc)] + [_vp] * 6 + [_sz, _vp]),
            "moe_grad_scratch_bytes": (_sz, [_i32]),
            "moe_grad_norm": (_i32, [ctypes.POINTER(moe_grad), _i32, _vp, _vp, _sz, _vp]),
            "moe_grad_clip": (_i32, [ctypes.POINTER(moe_grad), _i32, _vp, ctypes.c_float, _vp]),
            "moe_check": (_i32, [_dp, _vp, _sz, _vp]),
            "moe_strerror": (ctypes.c_char_p, [_i32]),
            "moe_abi_version": (_i32, []),
            "moe_profile_enable": (_i32, [_i32]),
            "moe_profile_collect": (_i32, []),
            "moe_profile_get": (_i32, [_i32, ctypes.POINTER(ctypes.c_char_p),
                                       ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_i64)]),
            "moe_profile_reset": (_i32, []),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _lib = L
    return _lib


def _p(t):
    """Device address of a tensor (or None), as a ctypes pointer."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:  # the raw handle: building a torch Stream object takes 3 us a call
        import torch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def make_desc(T, D, F, E, K, mode=MOE_BF16, flags=0) -> moe_desc:
    return moe_desc(T, D, F, E, K, mode, flags)


def strerror(code: int) -> str:
    return lib().moe_strerror(code).decode()


def abi_version() -> int:
    return lib().moe_abi_version()


def moe_scratch_bytes(desc: moe_desc) -> int:
    return lib().moe_scratch_bytes(ctypes.byref(desc))


def moe_wprep_bytes(desc: moe_desc) -> int:
    return lib().moe_wprep_bytes(ctypes.byref(desc))


def moe_prepare_weights(desc, w1, w2, wprep, stream=None) -> int:
    return lib().moe_prepare_weights(ctypes.byref(desc), _p(w1), _p(w2), _p(wprep),
                                     0 if wprep is None else _nbytes(wprep), _stream(stream))


def moe_route(desc, topk_idx, scratch, stream=None) -> int:
    return lib().moe_route(ctypes.byref(desc), _p(topk_idx), _p(scratch), _nbytes(scratch),
                           _stream(stream))


def moe_router_fwd(desc, logits, topk_idx, topk_w, stream=None) -> int:
    return lib().moe_router_fwd(ctypes.byref(desc), _p(logits), _p(topk_idx), _p(topk_w),
                                _stream(stream))


def moe_router_bwd(desc, topk_idx, topk_w, dtopk_w, dlogits, stream=None) -> int:
    return lib().moe_router_bwd(ctypes.byref(desc), _p(topk_idx), _p(topk_w), _p(dtopk_w),
                                _p(dlogits), _stream(stream))


_look = None


def _lookups() -> tuple:
    """What the operators beside the layer look up in torch, once: (functions for the current GPU and its
    stream's raw handle, fp32, int32, masks, codes, values by moe_type)"""
    global _look
    import torch
    torch.cuda.current_device()  # raises where there is no GPU
    f32 = (torch.float32,)
    _look = (torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream, f32, (torch.int32,),
             (torch.uint8, torch.bool), (torch.uint8, torch.float8_e4m3fn),
             {MOE_TYPE_F32: f32, MOE_TYPE_BF16: (torch.bfloat16,)})
    return _look


def _addresses(dev: int, *tensors):
    """The device addresses of (tensor, element types, count) for contiguous tensors on GPU `dev`, the current
    one, of one of those types with that many elements at least (count None: _rows_fit has seen to it); None
    where one does not fit.  None and raw addresses go through: they are the C side's to check."""
    out = []
    for t, types, n in tensors:
        if t is None or t.__class__ is int:
            out.append(t)
        elif t.dtype in types and t.get_device() == dev and (n is None or t.numel() >= n and t.is_contiguous()):
            out.append(t.data_ptr())
        else:
            return None
    return out


def _rows_fit(t, rows: int, cols: int, ld: int) -> bool:
    """Whether a tensor has that many rows and columns, ld elements between its rows."""
    if t is None or t.__class__ is int:
        return True
    size, stride = t.shape, t.stride()
    return len(size) == 2 and size[0] >= rows and size[1] >= cols and \
        (rows <= 1 or stride[0] == ld) and (cols <= 1 or stride[1] == 1)


def _scratch(t, dev: int) -> tuple:
    """(address, bytes) of a scratch tensor on GPU `dev`; (None, 0) where it does not fit or is None."""
    if t is None or t.get_device() != dev or not t.is_contiguous():
        return None, 0
    return t.data_ptr(), t.nbytes


def moe_balance_scratch_bytes(desc: moe_desc) -> int:
    return lib().moe_balance_scratch_bytes(ctypes.byref(desc))


def moe_balance_fwd(desc, logits, topk_idx, valid, counts, mean_p, losses, scratch, stream=None) -> int:
    T, E, K = desc.T, desc.E, desc.K
    device, raw, f32, i32, mask, _, _ = _look or _lookups()
    dev = device()
    at = _addresses(dev, (logits, f32, T * E), (topk_idx, i32, T * K), (valid, mask, T), (counts, i32, E + 1),
                    (mean_p, f32, E), (losses, f32, 2))
    if at is None:
        return MOE_EINVAL
    return lib().moe_balance_fwd(ctypes.byref(desc), *at, *_scratch(scratch, dev),
                                 raw(dev) if stream is None else _stream(stream))


def moe_balance_bwd(desc, logits, valid, counts, dlosses, topk_idx, topk_w, dtopk_w, dlogits,
                    stream=None) -> int:
    T, E, K = desc.T, desc.E, desc.K
    device, raw, f32, i32, mask, _, _ = _look or _lookups()
    dev = device()
    at = _addresses(dev, (logits, f32, T * E), (valid, mask, T), (counts, i32, E + 1), (dlosses, f32, 2),
                    (topk_idx, i32, T * K), (topk_w, f32, T * K), (dtopk_w, f32, T * K), (dlogits, f32, T * E))
    if at is None:
        return MOE_EINVAL
    return lib().moe_balance_bwd(ctypes.byref(desc), *at, raw(dev) if stream is None else _stream(stream))


def _code_ld(n: int) -> int:
    return (n + 15) // 16 * 16


def make_block_quant_desc(rows, cols, in_type=MOE_TYPE_BF16, scale=MOE_SCALE_TILE, ld_in=None,
                          ld_codes=None, ld_codes_t=None) -> moe_block_quant_desc:
    """Row strides default to the columns; those of codes to their next multiple of 16."""
    return moe_block_quant_desc(rows, cols, in_type, scale, cols if ld_in is None else ld_in,
                                _code_ld(cols) if ld_codes is None else ld_codes,
                                _code_ld(rows) if ld_codes_t is None else ld_codes_t)


def moe_block_quant(desc, x, codes, scales, codes_t=None, scales_t=None, stream=None) -> int:
    R, C = desc.rows, desc.cols
    rb, cb = (R + 127) // 128, (C + 127) // 128
    block = desc.scale == MOE_SCALE_BLOCK
    device, raw, f32, _, _, code, io = _look or _lookups()
    dev = device()
    if not (_rows_fit(x, R, C, desc.ld_in) and _rows_fit(codes, R, _code_ld(C), desc.ld_codes)
            and _rows_fit(codes_t, C, _code_ld(R), desc.ld_codes_t)):
        return MOE_EINVAL
    at = _addresses(dev, (x, io.get(desc.in_type, ()), None), (codes, code, None),
                    (scales, f32, cb * (rb if block else R)), (codes_t, code, None),
                    (scales_t, f32, rb * (cb if block else C)))
    if at is None:
        return MOE_EINVAL
    return lib().moe_block_quant(ctypes.byref(desc), *at, raw(dev) if stream is None else _stream(stream))


def make_block_mm_desc(M, N, K, a_type=MOE_TYPE_E4M3, b_scale=MOE_SCALE_BLOCK, c_type=MOE_TYPE_BF16,
                       flags=0, lda=None, ldb=None, ldc=None) -> moe_block_mm_desc:
    """Row strides as in make_block_quant_desc."""
    if lda is None:
        lda = _code_ld(K) if a_type == MOE_TYPE_E4M3 else K
    return moe_block_mm_desc(M, N, K, a_type, b_scale, c_type, flags, lda,
                             _code_ld(K) if ldb is None else ldb, N if ldc is None else ldc)


def moe_block_mm_scratch_bytes(desc: moe_block_mm_desc) -> int:
    return lib().moe_block_mm_scratch_bytes(ctypes.byref(desc))


def moe_block_mm(desc, a, a_scales, b, b_scales, c, scratch=None, stream=None) -> int:
    M, N, K = desc.M, desc.N, desc.K
    steps, own = (K + 127) // 128, desc.a_type == MOE_TYPE_E4M3
    device, raw, f32, _, _, code, io = _look or _lookups()
    dev = device()
    ldk = _code_ld(K)
    if not (_rows_fit(a, M, ldk if own else K, desc.lda) and _rows_fit(b, N, ldk, desc.ldb)
            and _rows_fit(c, M, N, desc.ldc)):
        return MOE_EINVAL
    at = _addresses(dev, (a, code if own else io.get(desc.a_type, ()), None), (a_scales, f32, steps * M),
                    (b, code, None),
                    (b_scales, f32, steps * (N if desc.b_scale == MOE_SCALE_TILE else (N + 127) // 128)),
                    (c, io.get(desc.c_type, ()), None))
    if at is None:
        return MOE_EINVAL
    return lib().moe_block_mm(ctypes.byref(desc), *at, *_scratch(scratch, dev),
                              raw(dev) if stream is None else _stream(stream))


def make_grad_list(src, dst=None):
    """The moe_grad array of contiguous GPU tensors (float32 or bfloat16) and of where their clipped
    values go (default: in place).  It holds addresses: keep the tensors alive, and make it anew when
    they move.  The calls that take it refuse it with another GPU current than the tensors'."""
    import torch
    types = {torch.float32: MOE_TYPE_F32, torch.bfloat16: MOE_TYPE_BF16}
    src = list(src)
    dst = src if dst is None else list(dst)
    if len(dst) != len(src):
        raise ValueError("as many destinations as gradients")
    for s, d in zip(src, dst):
        if s.dtype not in types or d.dtype != s.dtype or d.numel() != s.numel():
            raise ValueError("gradients are float32 or bfloat16, their destinations alike")
        if not (s.is_cuda and d.device == s.device == src[0].device and s.is_contiguous() and d.is_contiguous()):
            raise ValueError("gradients and destinations are contiguous tensors on one GPU")
    grads = (moe_grad * len(src))(*[moe_grad(s.data_ptr(), d.data_ptr(), s.numel(), types[s.dtype], 0)
                                    for s, d in zip(src, dst)])
    grads.device = src[0].get_device() if src else None
    return grads


def moe_grad_scratch_bytes(count: int) -> int:
    return lib().moe_grad_scratch_bytes(count)


def moe_grad_norm(grads, norm, scratch, stream=None) -> int:
    device, raw, f32, *_ = _look or _lookups()
    dev = device()
    at = _addresses(dev, (norm, f32, 1))
    if at is None or getattr(grads, "device", dev) not in (dev, None):
        return MOE_EINVAL
    return lib().moe_grad_norm(grads, len(grads), *at, *_scratch(scratch, dev),
                               raw(dev) if stream is None else _stream(stream))


def moe_grad_clip(grads, norm, max_norm: float, stream=None) -> int:
    device, raw, f32, *_ = _look or _lookups()
    dev = device()
    at = _addresses(dev, (norm, f32, 1))
    if at is None or getattr(grads, "device", dev) not in (dev, None):
        return MOE_EINVAL
    return lib().moe_grad_clip(grads, len(grads), *at, max_norm, raw(dev) if stream is None else _stream(stream))


def moe_routing_view(desc, scratch) -> tuple:
    """(status, counts, offsets, pos, src) device addresses inside scratch."""
    out = [_vp() for _ in range(4)]
    rc = lib().moe_routing_view(ctypes.byref(desc), _p(scratch), _nbytes(scratch),
                                *[ctypes.byref(o) for o in out])
    return (rc, *[o.value for o in out])


def moe_scratch_view(desc, scratch, which: int) -> tuple:
    """(status, device address, bytes) of an intermediate inside scratch."""
    ptr, n = _vp(), _sz()
    rc = lib().moe_scratch_view(ctypes.byref(desc), _p(scratch), _nbytes(scratch), which,
                                ctypes.byref(ptr), ctypes.byref(n))
    return rc, ptr.value, n.value


def moe_fwd(desc, x, topk_idx, topk_w, w1, w2, wprep, y, scratch, stream=None) -> int:
    return lib().moe_fwd(ctypes.byref(desc), _p(x), _p(topk_idx), _p(topk_w), _p(w1), _p(w2),
                         _p(wprep), _p(y), _p(scratch), _nbytes(scratch), _stream(stream))


def moe_fwd_noalloc(desc, x, topk_idx, topk_w, w1, w2, wprep, y, stream=None) -> int:
    return lib().moe_fwd_noalloc(ctypes.byref(desc), _p(x), _p(topk_idx), _p(topk_w), _p(w1),
                                 _p(w2), _p(wprep), _p(y), _stream(stream))


def moe_bwd(desc, dy, topk_w, w1, w2, wprep, dx, dw1, dw2, dtopk_w, scratch, stream=None) -> int:
    return lib().moe_bwd(ctypes.byref(desc), _p(dy), _p(topk_w), _p(w1), _p(w2), _p(wprep),
                         _p(dx), _p(dw1), _p(dw2), _p(dtopk_w), _p(scratch), _nbytes(scratch),
                         _stream(stream))


def moe_check(desc, scratch, stream=None) -> int:
    return lib().moe_check(ctypes.byref(desc), _p(scratch), _nbytes(scratch), _stream(stream))


def moe_profile_enable(on: bool) -> int:
    return lib().moe_profile_enable(1 if on else 0)


def moe_profile_collect() -> dict:
    """{kernel name: (total ms, launches)} accumulated since the last reset."""
    L = lib()
    n = L.moe_profile_collect()
    if n < 0:
        raise MoeError(n, "moe_profile_collect")
    out = {}
    for i in range(n):
        name, ms, cnt = ctypes.c_char_p(), ctypes.c_double(), _i64()
        L.moe_profile_get(i, ctypes.byref(name), ctypes.byref(ms), ctypes.byref(cnt))
        out[name.value.decode()] = (ms.value, cnt.value)
    return out


def moe_profile_reset() -> int:
    return lib().moe_profile_reset()


def check(code: int, what: str = "moe") -> None:
    """Raise MoeError for a non-zero status."""
    if code != MOE_OK:
        raise MoeError(code, what)
