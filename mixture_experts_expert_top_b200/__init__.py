"""Python binding of libmoe_b200, the B200 (sm_100a) MoE expert-FFN layer.

Argument marshalling only: every function here passes torch tensors' device
pointers and sizes to the C entry point of the same name (include/moe.h) and
raises MoeError on a non-OK status. All computation runs in the library's
CUDA kernels. If the library is missing this module raises on first use; it
has no fallback of any kind.

The layer: top-k softmax routing -> permute (bucket by expert, gather) ->
grouped GEMM gate/up + SwiGLU -> grouped GEMM down -> weighted finalize, with
a router by scores and an RMS norm beside it
(InfiniLM PR #500 Qwen3-MoE report §2.2; FlashInfer PR #7196 analysis §1-§2).
"""

from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import struct
from typing import Optional

import torch

__all__ = [
    "MoeError", "Shape", "lib", "library_path", "FMT_BF16", "FMT_INT4_G128",
    "moe_workspace_size", "moe_permute_workspace_size", "moe_forward_host_workspace_size",
    "moe_route", "moe_permute", "moe_grouped_gemm_swiglu", "moe_grouped_gemm_down",
    "moe_finalize", "moe_forward", "moe_forward_host", "moe_dequant_int4",
    "moe_get_device_error", "moe_status_string", "moe_permute_noalloc", "moe_selftest_bounded_wait",
    "moe_forward_kernel_count", "moe_forward_gathers_in_gemm", "forward", "debug_bounds_library",
    "moe_mx_quantize", "moe_grouped_gemm_swiglu_mx", "moe_grouped_gemm_down_mx", "FMT_MXFP8", "FMT_MXFP4",
    "moe_forward_fused", "moe_forward_is_fused",
    "FMT_INT8", "Router", "moe_route_scored", "moe_rmsnorm", "moe_i8_quantize", "moe_grouped_gemm_swiglu_i8",
    "moe_grouped_gemm_down_i8", "moe_forward_scored",
    "EP_MAX_RANKS", "EpPeers", "moe_ep_count", "moe_ep_dispatch", "moe_ep_local_offsets", "moe_ep_combine",
    "ep_forward",
]

HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(HERE, "libmoe_b200.so")

FMT_BF16 = 0
FMT_INT4_G128 = 1
FMT_MXFP8 = 2
FMT_MXFP4 = 3
FMT_INT8 = 4

STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED",
          3: "MOE_ERR_WORKSPACE_TOO_SMALL", 4: "MOE_ERR_CUDA", 5: "MOE_ERR_DEVICE_FLAG"}


EP_MAX_RANKS = 8


class EpPeers(ctypes.Structure):
    """moe_ep_peers_t: every rank's expert-parallel buffers (device addresses)."""
    _fields_ = [("world", ctypes.c_int32), ("rank", ctypes.c_int32), ("capacity", ctypes.c_int32),
                ("counts", ctypes.c_void_p * EP_MAX_RANKS), ("recv_rows", ctypes.c_void_p * EP_MAX_RANKS),
                ("recv_src", ctypes.c_void_p * EP_MAX_RANKS), ("y_ret", ctypes.c_void_p * EP_MAX_RANKS),
                ("pairs", ctypes.c_int32 * EP_MAX_RANKS)]


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


class Shape(ctypes.Structure):
    """moe_shape_t: E routed experts and top_k routed slots per token, plus
    n_shared shared experts (experts E.. of the weight arrays, one extra slot
    each with weight 1)."""
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("top_k", ctypes.c_int32), ("fmt", ctypes.c_int32),
                ("n_shared", ctypes.c_int32)]

    @classmethod
    def of(cls, T, H, I, E, top_k, fmt=FMT_BF16, n_shared=0) -> "Shape":
        if isinstance(fmt, str):
            fmt = {"bf16": FMT_BF16, "int4_g128": FMT_INT4_G128, "mxfp8": FMT_MXFP8, "mxfp4": FMT_MXFP4,
                   "int8": FMT_INT8}[fmt]
        return cls(int(T), int(H), int(I), int(E), int(top_k), int(fmt), int(n_shared))

    @property
    def slots(self) -> int:
        return self.top_k + self.n_shared

    @property
    def experts(self) -> int:
        return self.E + self.n_shared


class Router(ctypes.Structure):
    """moe_router_t: how moe_route_scored turns router logits into experts and
    weights (softmax or sigmoid scores, expert groups, renormalisation, scale)."""
    _fields_ = [("logits", ctypes.c_int32), ("score", ctypes.c_int32), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("group_top", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("scale", ctypes.c_float)]

    @classmethod
    def of(cls, score="softmax", n_group=1, topk_group=1, group_top=1, renormalize=True, scale=1.0,
           logits="fp32") -> "Router":
        return cls({"fp32": 0, "bf16": 1}[logits], {"softmax": 0, "sigmoid": 1}[score], int(n_group), int(topk_group),
                   int(group_top), int(bool(renormalize)), float(scale))


_lib: Optional[ctypes.CDLL] = None
_debug_lib: Optional[ctypes.CDLL] = None
_use_debug = False


def lib() -> ctypes.CDLL:
    """The loaded library (libmoe_b200.so; inside `debug_bounds_library()`,
    the range-checking build libmoe_b200_debug.so)."""
    global _lib, _debug_lib
    if _use_debug:
        if _debug_lib is None:
            _debug_lib = _load(True)
        return _debug_lib
    if _lib is None:
        _lib = _load(False)
    return _lib


class debug_bounds_library:
    """Context manager: the entry points of this module call the build made
    with -DMOE_DEBUG_BOUNDS (perm-derived rows and expert offsets range-checked
    in the kernels, device error 4 on a bad one) while it is active."""

    def __enter__(self):
        global _use_debug
        self._prev = _use_debug
        _use_debug = True
        return lib()

    def __exit__(self, *exc):
        global _use_debug
        _use_debug = self._prev
        return False


def _load(debug_bounds: bool) -> ctypes.CDLL:
    from . import build as _build
    path = _build.LIB_DEBUG if debug_bounds else library_path
    if not _build.up_to_date(debug_bounds):
        # a missing or stale library is rebuilt from the sources (needs nvcc); never skipped
        try:
            _build.build(debug_bounds=debug_bounds)
        except Exception as e:      # noqa: BLE001 - re-raised with the path
            raise RuntimeError(f"{path} is missing or older than its sources and could not be "
                               f"built ({e}): build it with `python -m mixture_experts_expert_top_b200.build`")
    L = ctypes.CDLL(path)
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
    sp = ctypes.POINTER(Shape)
    rp = ctypes.POINTER(Router)
    sigs = {
        "moe_workspace_size": ([sp], sz),
        "moe_permute_workspace_size": ([sp], sz),
        "moe_forward_host_workspace_size": ([sp], sz),
        "moe_route": ([vp, sp, vp, vp, vp], ctypes.c_int),
        "moe_permute": ([vp, sp, vp, vp, vp, vp, vp, vp, vp, sz, vp], ctypes.c_int),
        "moe_grouped_gemm_swiglu": ([vp, vp, vp, vp, vp, sp, vp, vp], ctypes.c_int),
        "moe_grouped_gemm_down": ([vp, vp, vp, vp, sp, vp, vp], ctypes.c_int),
        "moe_finalize": ([vp, vp, vp, sp, vp, vp], ctypes.c_int),
        "moe_forward": ([vp, vp, vp, vp, vp, vp, sp, vp, vp, sz, vp], ctypes.c_int),
        "moe_forward_host": ([vp, vp, vp, vp, vp, vp, sp, vp, vp, sz, vp], ctypes.c_int),
        "moe_dequant_int4": ([vp, vp, i32, i32, vp, vp], ctypes.c_int),
        "moe_mx_quantize": ([vp, i32, i32, vp, vp, vp], ctypes.c_int),
        "moe_forward_fused": ([vp, vp, vp, vp, sp, vp, vp, sz, vp], ctypes.c_int),
        "moe_grouped_gemm_swiglu_mx": ([vp, vp, vp, vp, vp, vp, sp, vp, vp, vp], ctypes.c_int),
        "moe_grouped_gemm_down_mx": ([vp, vp, vp, vp, vp, sp, vp, vp], ctypes.c_int),
        "moe_permute_noalloc": ([vp, sp, vp, vp, vp, vp, vp, vp, vp], ctypes.c_int),
        "moe_get_device_error": ([ctypes.POINTER(ctypes.c_int32)], ctypes.c_int),
        "moe_selftest_bounded_wait": ([ctypes.c_int64, vp], ctypes.c_int),
        "moe_forward_kernel_count": ([sp], ctypes.c_int32),
        "moe_forward_gathers_in_gemm": ([sp], ctypes.c_int32),
        "moe_forward_is_fused": ([sp], ctypes.c_int32),
        "moe_ep_count": ([vp, sp, ctypes.POINTER(EpPeers), vp], ctypes.c_int),
        "moe_ep_dispatch": ([vp, vp, vp, sp, ctypes.POINTER(EpPeers), vp], ctypes.c_int),
        "moe_ep_local_offsets": ([sp, ctypes.POINTER(EpPeers), vp, vp], ctypes.c_int),
        "moe_ep_combine": ([vp, vp, sp, ctypes.POINTER(EpPeers), vp], ctypes.c_int),
        "moe_route_scored": ([vp, vp, rp, sp, vp, vp, vp], ctypes.c_int),
        "moe_rmsnorm": ([vp, vp, vp, ctypes.c_float, i32, i32, i32, vp, vp, vp, vp, vp], ctypes.c_int),
        "moe_i8_quantize": ([vp, i32, i32, vp, vp, vp], ctypes.c_int),
        "moe_grouped_gemm_swiglu_i8": ([vp, vp, vp, vp, vp, vp, sp, vp, vp], ctypes.c_int),
        "moe_grouped_gemm_down_i8": ([vp, vp, vp, vp, vp, sp, vp, vp], ctypes.c_int),
        "moe_forward_scored": ([vp, vp, vp, rp, vp, vp, vp, vp, sp, vp, vp, sz, vp], ctypes.c_int),
        "moe_status_string": ([ctypes.c_int], ctypes.c_char_p),
    }
    for name, (args, res) in sigs.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    return L


# ---- marshalling helpers ---------------------------------------------------

BF16, F32, I32, U8, I8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.int8


def _p(t, *dtypes) -> Optional[int]:
    """Device (or host) address of a tensor, None for None. With dtypes, a
    tensor of another dtype is refused (the C ABI takes untyped pointers)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if dtypes and t.dtype not in dtypes:
        raise TypeError(f"libmoe_b200: expected a tensor of {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmoe_b200 must be contiguous")
    return t.data_ptr()


# element types as marshal.cpp has them (c10::ScalarType codes)
_U8, _I8, _I32, _F32, _BF16 = 0, 1, 3, 6, 15
_DTYPES = {_U8: U8, _I8: I8, _I32: I32, _F32: F32, _BF16: BF16}


def _addresses(dev: int, *spec):
    """Addresses of tensors given as (tensor, elements, type code) triples: each
    contiguous, of that type, with at least that many elements, on CUDA device
    dev; anything else (a host tensor, one of another device, a short one) is
    refused before the library is called. None and addresses (int) pass as they
    are. The checks run in _marshal; this function loads it and, on a refusal,
    says what is wrong."""
    global _checked
    if _checked is _addresses:
        from . import build as _build
        if not _build.marshal_up_to_date():
            try:
                _build.build_marshal()
            except Exception as e:      # noqa: BLE001 - re-raised with the path
                raise RuntimeError(f"{_build.marshal_file()} is missing or older than its source and could not be "
                                   f"built ({e}): build it with `python -m mixture_experts_expert_top_b200.build`")
        loader = importlib.machinery.ExtensionFileLoader(f"{__name__}._marshal", _build.marshal_file())
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader(loader.name, loader))
        loader.exec_module(module)
        _checked = module.addresses
    found = _checked(dev, *spec)
    if found is not None:
        return found
    given = [x for x in zip(spec[::3], spec[1::3], spec[2::3]) if x[0] is not None and x[0].__class__ is not int]
    for t, n, code in given:
        if not isinstance(t, torch.Tensor) or t.dtype is not _DTYPES[code]:
            raise TypeError(f"libmoe_b200: expected a tensor of {_DTYPES[code]}, got {getattr(t, 'dtype', type(t))}")
    for t, n, code in given:
        if t.layout is not torch.strided or not t.is_contiguous():
            raise ValueError("tensors passed to libmoe_b200 must be contiguous")
        if t.numel() < n:
            raise ValueError(f"libmoe_b200: expected at least {n} elements, got a tensor of shape {tuple(t.shape)}")
    for t, n, code in given:
        if t.get_device() != dev:
            raise ValueError(f"libmoe_b200: expected a tensor on the current CUDA device, got one on {t.device}")
    raise RuntimeError("libmoe_b200: a tensor was refused")


_checked = _addresses          # the _marshal module's from the first call on

# by format, per weight row of K elements: codes, scales, and their types
_WEIGHT_ROWS = {FMT_BF16: (lambda K: K, lambda K: 0, _BF16, _BF16),
                FMT_INT4_G128: (lambda K: K // 2, lambda K: K // 128, _U8, _BF16),
                FMT_MXFP8: (lambda K: K, lambda K: K // 32, _U8, _U8),
                FMT_MXFP4: (lambda K: K // 2, lambda K: K // 32, _U8, _U8),
                FMT_INT8: (lambda K: K, lambda K: 1, _I8, _F32)}


def _weights(shape: Shape, w_gu, w_gu_scales, w_d, w_d_scales):
    """The layer's weights as _addresses takes them."""
    _, H, I, E, _, fmt, S = _dims(shape)
    codes, scales, w_type, s_type = _WEIGHT_ROWS[fmt]
    gu, dn = (E + S) * 2 * I, (E + S) * H
    return (w_gu, gu * codes(H), w_type, w_gu_scales, gu * scales(H), s_type,
            w_d, dn * codes(I), w_type, w_d_scales, dn * scales(I), s_type)


_cuda_used = False


def _dev() -> int:
    """Index of the current CUDA device (-2 while this process has not used CUDA:
    then no tensor is on one)."""
    global _cuda_used
    if not _cuda_used:
        _cuda_used = torch.cuda.is_initialized()
        if not _cuda_used:
            return -2
    return torch._C._cuda_getDevice()


def _s(stream, dev: Optional[int] = None) -> Optional[int]:
    """A stream's handle; None is the current stream (of device dev, the current
    one). torch.cuda.current_stream() would build a Stream object, which takes
    longer (3.3 us) than a kernel's launch."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if dev is None or dev < 0 else dev)
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dims(shape: Shape):
    """(T, H, I, E, top_k, fmt, n_shared) of a shape."""
    return struct.unpack_from("7i", shape)


def _check(status: int, where: str) -> None:
    if status != 0:
        raise MoeError(status, where)


def _shape(shape) -> Shape:
    if isinstance(shape, Shape):
        return shape
    return Shape.of(*shape)


# ---- entry points (same names as the C ABI) --------------------------------

def moe_workspace_size(shape) -> int:
    return int(lib().moe_workspace_size(ctypes.byref(_shape(shape))))


def moe_permute_workspace_size(shape) -> int:
    return int(lib().moe_permute_workspace_size(ctypes.byref(_shape(shape))))


def moe_forward_host_workspace_size(shape) -> int:
    return int(lib().moe_forward_host_workspace_size(ctypes.byref(_shape(shape))))


def moe_route(logits, shape, topk_ids, topk_w, stream=None) -> None:
    _check(lib().moe_route(_p(logits, F32), ctypes.byref(_shape(shape)), _p(topk_ids, I32), _p(topk_w, F32),
                           _s(stream)),
           "moe_route")


def moe_route_scored(logits, bias, router: Router, shape, topk_ids, topk_w, stream=None) -> None:
    sh, d = _shape(shape), _dev()
    T, _, _, E, k, _, S = _dims(sh)
    n = T * (k + S)
    spec = (logits, T * E, _BF16 if router.logits else _F32, bias, E, _F32, topk_ids, n, _I32, topk_w, n, _F32)
    lg, b, ids, w = _checked(d, *spec) or _addresses(d, *spec)
    _check(lib().moe_route_scored(lg, b, router, sh, ids, w, _s(stream, d)), "moe_route_scored")


def moe_rmsnorm(x, residual, weight, eps: float, rows: int, H: int, fmt, residual_out, y, q=None, scales=None,
                stream=None) -> None:
    n, d = rows * H, _dev()
    q_type, s_type, n_scales = (_I8, _F32, rows) if fmt == FMT_INT8 else (_U8, _U8, n // 32)
    spec = (x, n, _BF16, residual, n, _BF16, weight, H, _BF16, residual_out, n, _BF16, y, n, _BF16, q, n, q_type,
            scales, n_scales, s_type)
    px, pr, pw, po, py, pq, ps = _checked(d, *spec) or _addresses(d, *spec)
    _check(lib().moe_rmsnorm(px, pr, pw, eps, rows, H, fmt, po, py, pq, ps, _s(stream, d)), "moe_rmsnorm")


def moe_permute(topk_ids, shape, counts, offsets, perm, inv_perm, hidden=None, hidden_perm=None,
                ws=None, stream=None) -> None:
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().moe_permute(_p(topk_ids, I32), ctypes.byref(_shape(shape)), _p(counts, I32), _p(offsets, I32),
                             _p(perm, I32), _p(inv_perm, I32), _p(hidden, BF16), _p(hidden_perm, BF16), _p(ws),
                             nbytes, _s(stream)),
           "moe_permute")


def moe_permute_noalloc(topk_ids, shape, counts, offsets, perm, inv_perm, hidden=None, hidden_perm=None,
                        stream=None) -> None:
    """moe_permute without a workspace: its scratch is a fixed array inside the
    library (for callers that cannot allocate device memory)."""
    _check(lib().moe_permute_noalloc(_p(topk_ids, I32), ctypes.byref(_shape(shape)), _p(counts, I32),
                                     _p(offsets, I32), _p(perm, I32), _p(inv_perm, I32), _p(hidden, BF16),
                                     _p(hidden_perm, BF16), _s(stream)),
           "moe_permute_noalloc")


def moe_grouped_gemm_swiglu(a, perm, offsets, w_gu, w_gu_scales, shape, act, stream=None) -> None:
    _check(lib().moe_grouped_gemm_swiglu(_p(a, BF16), _p(perm, I32), _p(offsets, I32), _p(w_gu, BF16, U8),
                                         _p(w_gu_scales, BF16, U8), ctypes.byref(_shape(shape)), _p(act, BF16),
                                         _s(stream)),
           "moe_grouped_gemm_swiglu")


def moe_grouped_gemm_down(act, offsets, w_d, w_d_scales, shape, y, stream=None) -> None:
    _check(lib().moe_grouped_gemm_down(_p(act, BF16), _p(offsets, I32), _p(w_d, BF16, U8), _p(w_d_scales, BF16, U8),
                                       ctypes.byref(_shape(shape)), _p(y, BF16), _s(stream)),
           "moe_grouped_gemm_down")


def moe_finalize(y, topk_w, inv_perm, shape, out, stream=None) -> None:
    _check(lib().moe_finalize(_p(y, BF16), _p(topk_w, F32), _p(inv_perm, I32), ctypes.byref(_shape(shape)),
                              _p(out, BF16), _s(stream)),
           "moe_finalize")


def moe_forward(hidden, logits, w_gu, w_gu_scales, w_d, w_d_scales, shape, out, ws, stream=None) -> None:
    nbytes, sh = ws.numel() * ws.element_size(), _shape(shape)
    if sh.fmt == FMT_INT8:
        d = _dev()
        spec = (hidden, sh.T * sh.H, _BF16, logits, sh.T * sh.E, _F32, *_weights(sh, w_gu, w_gu_scales, w_d, w_d_scales),
                out, sh.T * sh.H, _BF16)
        ph, pl, pg, pgs, pd, pds, po = _checked(d, *spec) or _addresses(d, *spec)
    else:
        ph, pl, pg, pgs = _p(hidden, BF16), _p(logits, F32), _p(w_gu, BF16, U8), _p(w_gu_scales, BF16, U8)
        pd, pds, po = _p(w_d, BF16, U8), _p(w_d_scales, BF16, U8), _p(out, BF16)
    _check(lib().moe_forward(ph, pl, pg, pgs, pd, pds, ctypes.byref(sh), po, _p(ws), nbytes, _s(stream)), "moe_forward")


def moe_forward_host(hidden_host, logits_host, w_gu, w_gu_scales, w_d, w_d_scales, shape, out_host, ws,
                     stream=None) -> None:
    nbytes, sh = ws.numel() * ws.element_size(), _shape(shape)
    if sh.fmt == FMT_INT8:
        d = _dev()
        spec = _weights(sh, w_gu, w_gu_scales, w_d, w_d_scales)
        pg, pgs, pd, pds = _checked(d, *spec) or _addresses(d, *spec)
    else:
        pg, pgs = _p(w_gu, BF16, U8), _p(w_gu_scales, BF16, U8)
        pd, pds = _p(w_d, BF16, U8), _p(w_d_scales, BF16, U8)
    _check(lib().moe_forward_host(_p(hidden_host, BF16), _p(logits_host, F32), pg, pgs, pd, pds, ctypes.byref(sh),
                                  _p(out_host, BF16), _p(ws), nbytes, _s(stream)),
           "moe_forward_host")


def moe_forward_fused(hidden, logits, w_gu, w_d, shape, out, ws, stream=None) -> None:
    nbytes = ws.numel() * ws.element_size()
    _check(lib().moe_forward_fused(_p(hidden, BF16), _p(logits, F32), _p(w_gu, BF16), _p(w_d, BF16),
                                   ctypes.byref(_shape(shape)), _p(out, BF16), _p(ws), nbytes, _s(stream)),
           "moe_forward_fused")


def moe_mx_quantize(x, rows: int, K: int, q, scales, stream=None) -> None:
    _check(lib().moe_mx_quantize(_p(x, BF16), int(rows), int(K), _p(q, U8), _p(scales, U8), _s(stream)),
           "moe_mx_quantize")


def moe_grouped_gemm_swiglu_mx(a_q, a_scales, perm, offsets, w_gu, w_gu_scales, shape, act_q, act_scales,
                               stream=None) -> None:
    _check(lib().moe_grouped_gemm_swiglu_mx(_p(a_q, U8), _p(a_scales, U8), _p(perm, I32), _p(offsets, I32),
                                            _p(w_gu, U8), _p(w_gu_scales, U8), ctypes.byref(_shape(shape)),
                                            _p(act_q, U8), _p(act_scales, U8), _s(stream)),
           "moe_grouped_gemm_swiglu_mx")


def moe_grouped_gemm_down_mx(act_q, act_scales, offsets, w_d, w_d_scales, shape, y, stream=None) -> None:
    _check(lib().moe_grouped_gemm_down_mx(_p(act_q, U8), _p(act_scales, U8), _p(offsets, I32), _p(w_d, U8),
                                          _p(w_d_scales, U8), ctypes.byref(_shape(shape)), _p(y, BF16), _s(stream)),
           "moe_grouped_gemm_down_mx")


def moe_i8_quantize(x, rows: int, K: int, q, scales, stream=None) -> None:
    n, d = rows * K, _dev()
    spec = (x, n, _BF16, q, n, _I8, scales, rows, _F32)
    px, pq, ps = _checked(d, *spec) or _addresses(d, *spec)
    _check(lib().moe_i8_quantize(px, rows, K, pq, ps, _s(stream, d)), "moe_i8_quantize")


def moe_grouped_gemm_swiglu_i8(a_q, a_scales, perm, offsets, w_gu, w_gu_scales, shape, act, stream=None) -> None:
    sh, d = _shape(shape), _dev()
    T, H, I, E, k, _, S = _dims(sh)
    P, E = T * (k + S), E + S
    rows = P if perm is None else T
    spec = (a_q, rows * H, _I8, a_scales, rows, _F32, perm, P, _I32, offsets, E + 1, _I32, w_gu, E * 2 * I * H, _I8,
            w_gu_scales, E * 2 * I, _F32, act, P * I, _BF16)
    pa, ps, pp, po, pw, pg, pc = _checked(d, *spec) or _addresses(d, *spec)
    _check(lib().moe_grouped_gemm_swiglu_i8(pa, ps, pp, po, pw, pg, sh, pc, _s(stream, d)), "moe_grouped_gemm_swiglu_i8")


def moe_grouped_gemm_down_i8(act_q, act_scales, offsets, w_d, w_d_scales, shape, y, stream=None) -> None:
    sh, d = _shape(shape), _dev()
    T, H, I, E, k, _, S = _dims(sh)
    P, E = T * (k + S), E + S
    spec = (act_q, P * I, _I8, act_scales, P, _F32, offsets, E + 1, _I32, w_d, E * H * I, _I8, w_d_scales, E * H, _F32,
            y, P * H, _BF16)
    pa, ps, po, pw, pg, py = _checked(d, *spec) or _addresses(d, *spec)
    _check(lib().moe_grouped_gemm_down_i8(pa, ps, po, pw, pg, sh, py, _s(stream, d)), "moe_grouped_gemm_down_i8")


def moe_forward_scored(hidden, logits, bias, router: Router, w_gu, w_gu_scales, w_d, w_d_scales, shape, out, ws,
                       stream=None) -> None:
    sh, d = _shape(shape), _dev()
    T, H, _, E, _, fmt, _ = _dims(sh)
    if fmt not in _WEIGHT_ROWS:
        raise MoeError(1, "moe_forward_scored")
    if ws.dtype is not U8:
        if not ws.is_contiguous():
            raise ValueError("tensors passed to libmoe_b200 must be contiguous")
        ws = ws.unsqueeze(0).view(U8)
    spec = (hidden, T * H, _BF16, logits, T * E, _BF16 if router.logits else _F32, bias, E, _F32,
            *_weights(sh, w_gu, w_gu_scales, w_d, w_d_scales), out, T * H, _BF16, ws, 0, _U8)
    ph, pl, pb, pg, pgs, pd, pds, po, pws = _checked(d, *spec) or _addresses(d, *spec)
    _check(lib().moe_forward_scored(ph, pl, pb, router, pg, pgs, pd, pds, sh, po, pws, ws.numel(), _s(stream, d)),
           "moe_forward_scored")


def moe_dequant_int4(q, scales, rows: int, K: int, out, stream=None) -> None:
    _check(lib().moe_dequant_int4(_p(q, U8), _p(scales, BF16), int(rows), int(K), _p(out, BF16), _s(stream)),
           "moe_dequant_int4")


def moe_forward_kernel_count(shape) -> int:
    return int(lib().moe_forward_kernel_count(ctypes.byref(_shape(shape))))


def moe_forward_is_fused(shape) -> bool:
    v = int(lib().moe_forward_is_fused(ctypes.byref(_shape(shape))))
    if v < 0:
        raise MoeError(1, "moe_forward_is_fused: invalid shape")
    return v == 1


def moe_forward_gathers_in_gemm(shape) -> bool:
    v = int(lib().moe_forward_gathers_in_gemm(ctypes.byref(_shape(shape))))
    if v < 0:
        raise MoeError(1, "moe_forward_gathers_in_gemm: invalid shape")
    return v == 1


def moe_selftest_bounded_wait(limit_ns: int, stream=None) -> None:
    _check(lib().moe_selftest_bounded_wait(int(limit_ns), _s(stream)), "moe_selftest_bounded_wait")


def moe_get_device_error() -> int:
    code = ctypes.c_int32(0)
    _check(lib().moe_get_device_error(ctypes.byref(code)), "moe_get_device_error")
    return int(code.value)


def moe_status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


# ---- convenience -----------------------------------------------------------

def forward(hidden: torch.Tensor, logits: torch.Tensor, w_gu: torch.Tensor, w_d: torch.Tensor, top_k: int,
            w_gu_scales: Optional[torch.Tensor] = None, w_d_scales: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None,
            router: Optional[Router] = None, bias: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_forward on device tensors; allocates out and the workspace with
    torch when they are not given. hidden [T,H] bf16, logits [T,E] fp32,
    w_gu [E+S,2I,H] bf16 (or uint8: int4 [E+S,2I,H/2] with bf16 scales, MXFP8
    [E+S,2I,H] or MXFP4 [E+S,2I,H/2] with uint8 scales; or int8 [E+S,2I,H] with
    fp32 scales [E+S,2I]), w_d likewise: weight arrays with more experts than
    logits columns hold S shared experts after the E routed ones. With a
    router, moe_forward_scored (logits fp32 or bf16 as the router says, bias
    [E] fp32 or None)."""
    T, H = hidden.shape
    E = logits.shape[1]
    if bias is not None and router is None:
        raise ValueError("a selection bias needs a router")
    if w_gu.dtype == torch.int8:
        fmt = FMT_INT8
    elif w_gu.dtype != torch.uint8:
        fmt = FMT_BF16
    elif w_gu_scales is None or w_gu_scales.dtype != torch.uint8:
        fmt = FMT_INT4_G128
    else:
        fmt = FMT_MXFP4 if w_gu.shape[2] * 2 == H else FMT_MXFP8
    I = w_d.shape[2] * (2 if fmt in (FMT_INT4_G128, FMT_MXFP4) else 1)
    shape = Shape.of(T, H, I, E, top_k, fmt, n_shared=w_gu.shape[0] - E)
    if out is None:
        out = torch.empty(T, H, dtype=torch.bfloat16, device=hidden.device)
    if ws is None:
        ws = torch.empty(max(moe_workspace_size(shape), 1), dtype=torch.uint8, device=hidden.device)
    if router is not None:
        moe_forward_scored(hidden, logits, bias, router, w_gu, w_gu_scales, w_d, w_d_scales, shape, out, ws, stream)
    else:
        moe_forward(hidden, logits, w_gu, w_gu_scales, w_d, w_d_scales, shape, out, ws, stream)
    return out


# ---- expert parallelism -----------------------------------------------------

def moe_ep_count(offsets, shape, peers: EpPeers, stream=None) -> None:
    _check(lib().moe_ep_count(_p(offsets, I32), ctypes.byref(_shape(shape)), ctypes.byref(peers), _s(stream)),
           "moe_ep_count")


def moe_ep_dispatch(hidden, perm, offsets, shape, peers: EpPeers, stream=None) -> None:
    _check(lib().moe_ep_dispatch(_p(hidden, BF16), _p(perm, I32), _p(offsets, I32), ctypes.byref(_shape(shape)),
                                 ctypes.byref(peers), _s(stream)), "moe_ep_dispatch")


def moe_ep_local_offsets(shape, peers: EpPeers, offsets_local, stream=None) -> None:
    _check(lib().moe_ep_local_offsets(ctypes.byref(_shape(shape)), ctypes.byref(peers), _p(offsets_local, I32),
                                      _s(stream)), "moe_ep_local_offsets")


def moe_ep_combine(y_local, offsets_local, shape, peers: EpPeers, stream=None) -> None:
    _check(lib().moe_ep_combine(_p(y_local, BF16), _p(offsets_local, I32), ctypes.byref(_shape(shape)),
                                ctypes.byref(peers), _s(stream)), "moe_ep_combine")


def ep_forward(ranks, w_gu_shards, w_d_shards, top_k: int, devices=None):
    """The layer with its experts split over len(ranks) ranks driven from one
    process: rank r holds tokens ranks[r] = (hidden [T_r,H] bf16, logits
    [T_r,E] fp32) and the weights of experts r*E/R .. (r+1)*E/R - 1
    (w_gu_shards[r] [E/R,2I,H], w_d_shards[r] [E/R,H,I], bf16), all on device
    devices[r] (default: the current device for every rank, i.e. R ranks
    emulated on one GPU; ranks on different GPUs need peer access between
    them). The phases (route and permute, count, dispatch, local GEMMs,
    combine, finalize) are separated by a synchronisation of every rank's
    device, the barrier moe_ep_peers_t's steps ask for. Returns each rank's
    out [T_r,H] bf16."""
    R = len(ranks)
    if not 1 <= R <= EP_MAX_RANKS:
        raise ValueError(f"1 <= ranks <= {EP_MAX_RANKS}")
    devs = [torch.device(d) for d in (devices or [torch.cuda.current_device()] * R)]
    H = ranks[0][0].shape[1]
    E = ranks[0][1].shape[1]
    E_loc, I = w_d_shards[0].shape[0], w_d_shards[0].shape[2]
    if E_loc * R != E:
        raise ValueError("the weight shards must split the E experts evenly")
    k = int(top_k)
    Ts = [int(h.shape[0]) for h, _ in ranks]
    capacity = ((sum(Ts) * k + k - 1) // k) * k          # every pair of every rank at one owner
    i32 = torch.int32
    st = []
    for r, (h, lg) in enumerate(ranks):
        d = devs[r]
        P = Ts[r] * k
        st.append({
            "shape": Shape.of(Ts[r], H, I, E, k),
            "ids": torch.empty(Ts[r], k, dtype=i32, device=d), "w": torch.empty(Ts[r], k, device=d),
            "counts_g": torch.empty(E, dtype=i32, device=d), "offsets": torch.empty(E + 1, dtype=i32, device=d),
            "perm": torch.empty(P, dtype=i32, device=d), "inv": torch.empty(P, dtype=i32, device=d),
            "counts": torch.zeros(R, E_loc, dtype=i32, device=d),
            "recv_rows": torch.empty(capacity, H, dtype=torch.bfloat16, device=d),
            "recv_src": torch.empty(capacity, dtype=i32, device=d),
            "y_ret": torch.empty(max(P, 1), H, dtype=torch.bfloat16, device=d),
            "off_loc": torch.empty(E_loc + 1, dtype=i32, device=d),
            "act": torch.empty(capacity, I, dtype=torch.bfloat16, device=d),
            "y_loc": torch.empty(capacity, H, dtype=torch.bfloat16, device=d),
            "out": torch.empty(Ts[r], H, dtype=torch.bfloat16, device=d),
            "pws": torch.empty(max(1, moe_permute_workspace_size(Shape.of(Ts[r], H, I, E, k))), dtype=torch.uint8,
                               device=d),
        })
    shape_loc = Shape.of(capacity // k, H, I, E_loc, k)

    def peers(r):
        pe = EpPeers()
        pe.world, pe.rank, pe.capacity = R, r, capacity
        for q in range(R):
            pe.counts[q] = st[q]["counts"].data_ptr()
            pe.recv_rows[q] = st[q]["recv_rows"].data_ptr()
            pe.recv_src[q] = st[q]["recv_src"].data_ptr()
            pe.y_ret[q] = st[q]["y_ret"].data_ptr()
            pe.pairs[q] = Ts[q] * k
        return pe

    def barrier():
        for d in set(devs):
            torch.cuda.synchronize(d)

    def each(fn):
        for r in range(R):
            with torch.cuda.device(devs[r]):
                fn(r)
        barrier()

    def route_permute(r):
        h, lg = ranks[r]
        s = st[r]
        moe_route(lg, s["shape"], s["ids"], s["w"])
        moe_permute(s["ids"], s["shape"], s["counts_g"], s["offsets"], s["perm"], s["inv"], None, None, s["pws"])

    def local_gemms(r):
        s = st[r]
        moe_ep_local_offsets(s["shape"], peers(r), s["off_loc"])
        moe_grouped_gemm_swiglu(s["recv_rows"], None, s["off_loc"], w_gu_shards[r], None, shape_loc, s["act"])
        moe_grouped_gemm_down(s["act"], s["off_loc"], w_d_shards[r], None, shape_loc, s["y_loc"])

    def finalize(r):
        s = st[r]
        ident = torch.arange(Ts[r] * k, dtype=i32, device=devs[r])
        moe_finalize(s["y_ret"], s["w"], ident, s["shape"], s["out"])

    each(route_permute)
    each(lambda r: moe_ep_count(st[r]["offsets"], st[r]["shape"], peers(r)))
    each(lambda r: moe_ep_dispatch(ranks[r][0], st[r]["perm"], st[r]["offsets"], st[r]["shape"], peers(r)))
    each(local_gemms)
    each(lambda r: moe_ep_combine(st[r]["y_loc"], st[r]["off_loc"], st[r]["shape"], peers(r)))
    each(finalize)
    return [s["out"] for s in st]
