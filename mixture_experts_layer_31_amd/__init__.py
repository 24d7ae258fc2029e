"""Python binding of the MI355X MoE layer's C ABI (include/moe.h).

Argument marshalling only: every step of the layer runs in the HIP library
libmoe_mi355x.so built in-tree by ``mixture_experts_layer_31_amd.build``.  The
functions below carry the C names; tensors are torch tensors on the GPU (or
None for optional pointers) and `stream` defaults to torch's current stream.
Loading fails loudly when the library has not been built: there is no fallback.
The calls of the operators beside the layer (moe_balance_*, moe_gate_*, moe_block_*,
moe_norm_*, moe_grad_*, moe_adamw) also look at their tensors: one of another type, device or stride than the call takes,
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
MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX = range(2)
MOE_GATE_RENORM, MOE_GATE_ACCUMULATE = 0x1, 0x2

# Exported symbols, in the order include/moe.h declares them.
EXPORTS = (
    "moe_scratch_bytes", "moe_wprep_bytes", "moe_prepare_weights", "moe_route",
    "moe_routing_view", "moe_scratch_view", "moe_fwd", "moe_bwd", "moe_fwd_noalloc", "moe_router_fwd",
    "moe_router_bwd", "moe_balance_scratch_bytes", "moe_balance_fwd", "moe_balance_bwd", "moe_gate_fwd", "moe_gate_bwd",
    "moe_gate_bias", "moe_block_quant", "moe_block_mm_scratch_bytes", "moe_block_mm", "moe_norm_fwd",
    "moe_norm_scratch_bytes", "moe_norm_bwd", "moe_grad_scratch_bytes", "moe_grad_norm", "moe_grad_clip",
    "moe_adamw", "moe_check", "moe_strerror", "moe_abi_version", "moe_profile_enable", "moe_profile_collect",
    "moe_profile_get", "moe_profile_reset",
)


class moe_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "D", "F", "E", "K", "mode", "flags")]


class moe_gate_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "E", "K", "groups", "top_groups", "group_best", "score", "in_type",
                                              "flags")] + \
               [("scale", ctypes.c_float)] + [(n, ctypes.c_int64) for n in ("ld_logits", "ld_dlogits")]


class moe_block_quant_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "cols", "in_type", "scale")] + \
               [(n, ctypes.c_int64) for n in ("ld_in", "ld_codes", "ld_codes_t")]


class moe_block_mm_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("M", "N", "K", "a_type", "b_scale", "c_type", "flags")] + \
               [(n, ctypes.c_int64) for n in ("lda", "ldb", "ldc")]


class moe_norm_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "D", "io_type", "res_type", "w_type")] + \
               [(n, ctypes.c_float) for n in ("eps", "scale")] + \
               [(n, ctypes.c_int64) for n in ("ld_b", "ld_r", "ld_h", "ld_y")]


class moe_grad(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("type", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class moe_adamw_param(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "master", "grad", "m", "v", "m_scale", "v_scale")] + \
               [("n", ctypes.c_int64), ("param_type", ctypes.c_int32), ("grad_type", ctypes.c_int32),
                ("weight_decay", ctypes.c_float), ("reserved", ctypes.c_int32)]


class moe_adamw_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("beta1", "beta2", "eps")] + \
               [("state_type", ctypes.c_int32), ("reserved", ctypes.c_int32)]


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
            "moe_gate_fwd": (_i32, [ctypes.POINTER(moe_gate_desc)] + [_vp] * 5),
            "moe_gate_bwd": (_i32, [ctypes.POINTER(moe_gate_desc)] + [_vp] * 5),
            "moe_gate_bias": (_i32, [_i32, _vp, ctypes.c_float, _vp, _vp]),
            "moe_block_quant": (_i32, [ctypes.POINTER(moe_block_quant_desc)] + [_vp] * 6),
            "moe_block_mm_scratch_bytes": (_sz, [ctypes.POINTER(moe_block_mm_desc)]),
            "moe_block_mm": (_i32, [ctypes.POINTER(moe_block_mm_desc)] + [_vp] * 6 + [_sz, _vp]),
            "moe_norm_fwd": (_i32, [ctypes.POINTER(moe_norm_desc)] + [_vp] * 8),
            "moe_norm_scratch_bytes": (_sz, [ctypes.POINTER(moe_norm_desc)]),
            "moe_norm_bwd": (_i32, [ctypes.POINTER(moe_norm_desc)] + [_vp] * 13 + [_sz, _vp]),
            "moe_grad_scratch_bytes": (_sz, [_i32]),
            "moe_grad_norm": (_i32, [ctypes.POINTER(moe_grad), _i32, _vp, _vp, _sz, _vp]),
            "moe_grad_clip": (_i32, [ctypes.POINTER(moe_grad), _i32, _vp, ctypes.c_float, _vp]),
            "moe_adamw": (_i32, [ctypes.POINTER(moe_adamw_desc), ctypes.POINTER(moe_adamw_param), _i32] + [_vp] * 3
                          + [ctypes.c_float, _vp]),
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


def make_gate_desc(T, E, K, score=MOE_SCORE_SIGMOID, groups=1, top_groups=1, group_best=2, in_type=MOE_TYPE_F32,
                   flags=MOE_GATE_RENORM, scale=1.0, ld_logits=None, ld_dlogits=None) -> moe_gate_desc:
    """Row strides default to the experts."""
    return moe_gate_desc(T, E, K, groups, top_groups, group_best, score, in_type, flags, scale,
                         E if ld_logits is None else ld_logits, E if ld_dlogits is None else ld_dlogits)


def moe_gate_fwd(desc, logits, bias, topk_idx, topk_w, stream=None) -> int:
    T, E, K = desc.T, desc.E, desc.K
    device, raw, f32, i32, _, _, io = _look or _lookups()
    dev = device()
    if not _rows_fit(logits, T, E, desc.ld_logits):
        return MOE_EINVAL
    at = _addresses(dev, (logits, io.get(desc.in_type, ()), None), (bias, f32, E), (topk_idx, i32, T * K),
                    (topk_w, f32, T * K))
    if at is None:
        return MOE_EINVAL
    return lib().moe_gate_fwd(ctypes.byref(desc), *at, raw(dev) if stream is None else _stream(stream))


def moe_gate_bwd(desc, logits, topk_idx, dtopk_w, dlogits, stream=None) -> int:
    T, E, K = desc.T, desc.E, desc.K
    device, raw, f32, i32, _, _, io = _look or _lookups()
    dev = device()
    if not (_rows_fit(logits, T, E, desc.ld_logits) and _rows_fit(dlogits, T, E, desc.ld_dlogits)):
        return MOE_EINVAL
    t = io.get(desc.in_type, ())
    at = _addresses(dev, (logits, t, None), (topk_idx, i32, T * K), (dtopk_w, f32, T * K), (dlogits, t, None))
    if at is None:
        return MOE_EINVAL
    return lib().moe_gate_bwd(ctypes.byref(desc), *at, raw(dev) if stream is None else _stream(stream))


def moe_gate_bias(counts, step: float, bias, stream=None) -> int:
    """One step of the bias [E]; counts [E] or longer (moe_balance_fwd's [E + 1])."""
    device, raw, f32, i32, *_ = _look or _lookups()
    dev = device()
    if bias is None:
        return MOE_EINVAL
    E = bias.numel()
    at = _addresses(dev, (counts, i32, E), (bias, f32, E))
    if at is None:
        return MOE_EINVAL
    return lib().moe_gate_bias(E, at[0], step, at[1], raw(dev) if stream is None else _stream(stream))


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


def make_norm_desc(T, D, io_type=MOE_TYPE_BF16, res_type=MOE_TYPE_BF16, w_type=MOE_TYPE_F32, eps=1e-6, scale=1.0,
                   ld_b=None, ld_r=None, ld_h=None, ld_y=None) -> moe_norm_desc:
    """Row strides default to the columns."""
    return moe_norm_desc(T, D, io_type, res_type, w_type, eps, scale, *[D if v is None else v
                                                                       for v in (ld_b, ld_r, ld_h, ld_y)])


def moe_norm_fwd(desc, b, r, gate, w_post, w, h, y, stream=None) -> int:
    T, D = desc.T, desc.D
    device, raw, f32, _, _, _, types = _look or _lookups()
    dev = device()
    if not (_rows_fit(b, T, D, desc.ld_b) and _rows_fit(r, T, D, desc.ld_r) and _rows_fit(h, T, D, desc.ld_h)
            and _rows_fit(y, T, D, desc.ld_y)):
        return MOE_EINVAL
    io, res, wt = types.get(desc.io_type, ()), types.get(desc.res_type, ()), types.get(desc.w_type, ())
    at = _addresses(dev, (b, io, None), (r, res, None), (gate, f32, T), (w_post, wt, D), (w, wt, D), (h, res, None),
                    (y, io, None))
    if at is None:
        return MOE_EINVAL
    return lib().moe_norm_fwd(ctypes.byref(desc), *at, raw(dev) if stream is None else _stream(stream))


def moe_norm_scratch_bytes(desc: moe_norm_desc) -> int:
    return lib().moe_norm_scratch_bytes(ctypes.byref(desc))


def moe_norm_bwd(desc, b, h, gate, w_post, w, dy, dh, db, dr, dgate, dw_post, dw, scratch, stream=None) -> int:
    T, D = desc.T, desc.D
    device, raw, f32, _, _, _, types = _look or _lookups()
    dev = device()
    if not (_rows_fit(b, T, D, desc.ld_b) and _rows_fit(h, T, D, desc.ld_h) and _rows_fit(dy, T, D, desc.ld_y)
            and _rows_fit(dh, T, D, desc.ld_h) and _rows_fit(db, T, D, desc.ld_b) and _rows_fit(dr, T, D, desc.ld_r)):
        return MOE_EINVAL
    io, res, wt = types.get(desc.io_type, ()), types.get(desc.res_type, ()), types.get(desc.w_type, ())
    at = _addresses(dev, (b, io, None), (h, res, None), (gate, f32, T), (w_post, wt, D), (w, wt, D), (dy, io, None),
                    (dh, res, None), (db, io, None), (dr, res, None), (dgate, f32, T), (dw_post, f32, D), (dw, f32, D))
    if at is None:
        return MOE_EINVAL
    return lib().moe_norm_bwd(ctypes.byref(desc), *at, *_scratch(scratch, dev),
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


def make_adamw_desc(beta1=0.9, beta2=0.95, eps=1e-8, state_type=MOE_TYPE_F32) -> moe_adamw_desc:
    return moe_adamw_desc(beta1, beta2, eps, state_type, 0)


def make_adamw_list(params, grads, m, v, masters=None, m_scales=None, v_scales=None, weight_decay=0.0):
    """The moe_adamw_param array of contiguous GPU tensors: params and grads float32 or bfloat16, the states
    float32, or uint8 or float8_e4m3fn codes with float32 scales ([ceil(n / 128)] each), masters float32 or None
    each, weight_decay a number or one a tensor.  It holds addresses: keep the tensors alive, and make it
    anew when they move.  The call refuses it with another GPU current than the tensors'."""
    import torch
    types = {torch.float32: MOE_TYPE_F32, torch.bfloat16: MOE_TYPE_BF16}
    params = list(params)
    count = len(params)
    e4m3 = m_scales is not None
    lists = [list(x) if x is not None else [None] * count for x in (masters, grads, m, v, m_scales, v_scales)]
    decay = [weight_decay] * count if isinstance(weight_decay, (int, float)) else list(weight_decay)
    if any(len(x) != count for x in (*lists, decay)) or (v_scales is not None) != e4m3:
        raise ValueError("as many of each as parameters; scales for both states or for none")
    codes = (torch.uint8, torch.float8_e4m3fn)
    rows = []
    for p, w, g, a, b, sa, sb, wd in zip(params, *lists, decay):
        n = p.numel()
        if p.dtype not in types or g is None or g.dtype not in types or g.numel() != n:
            raise ValueError("parameters and gradients are float32 or bfloat16, of one length")
        if w is not None and (p.dtype != torch.bfloat16 or w.dtype != torch.float32 or w.numel() != n):
            raise ValueError("a master is float32, beside a bfloat16 parameter of its length")
        if any(x is None or x.numel() < n or x.dtype not in (codes if e4m3 else (torch.float32,)) for x in (a, b)):
            raise ValueError("states have an element for each of the parameter's, float32 or codes")
        if e4m3 and any(x is None or x.dtype != torch.float32 or x.numel() < (n + 127) // 128 for x in (sa, sb)):
            raise ValueError("codes have a float32 scale for each 128")
        own = [x for x in (p, w, g, a, b, sa, sb) if x is not None]
        if not all(x.is_cuda and x.device == params[0].device and x.is_contiguous() for x in own):
            raise ValueError("contiguous tensors on one GPU")
        rows.append(moe_adamw_param(*[_p(x) for x in (p, w, g, a, b, sa, sb)], n, types[p.dtype], types[g.dtype], wd, 0))
    out = (moe_adamw_param * count)(*rows)
    out.device = params[0].get_device() if params else None
    out.state_type = MOE_TYPE_E4M3 if e4m3 else MOE_TYPE_F32
    return out


def moe_adamw(desc, params, lr, step, norm=None, max_norm: float = 0.0, stream=None) -> int:
    device, raw, f32, i32, *_ = _look or _lookups()
    dev = device()
    at = _addresses(dev, (lr, f32, 1), (step, i32, 1), (norm, f32, 1))
    if at is None or getattr(params, "device", dev) not in (dev, None) or \
            getattr(params, "state_type", desc.state_type) != desc.state_type:
        return MOE_EINVAL
    return lib().moe_adamw(ctypes.byref(desc), params, len(params), *at, max_norm,
                           raw(dev) if stream is None else _stream(stream))


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
