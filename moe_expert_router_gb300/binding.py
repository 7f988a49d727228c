"""ctypes binding of libmoe.so: the same entry points as include/moe.h.

Argument marshalling only -- every step of the expert path runs in the CUDA
kernels of libmoe. There is no fallback: if the library is missing or cannot be
loaded, every call raises.

Tensors are torch CUDA tensors; the stream defaults to torch's current stream
on the tensors' device.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

from .build import LIB_PATH, NATIVE_PATH

MOE_OK = 0
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED",
                3: "MOE_ERR_CUDA", 4: "MOE_ERR_WORKSPACE", 5: "MOE_ERR_DEVICE_FLAGGED"}
DEVERR_BAD_EXPERT_INDEX = 0x1
DEVERR_WAIT_TIMEOUT = 0x2
DEVERR_CAPACITY = 0x4
DEVERR_BAD_OFFSETS = 0x8
SCORE_SOFTMAX = 0
SCORE_SIGMOID = 1
SHAPE_TRAINING = 0x1
SHAPE_MXFP8 = 0x2
SHAPE_PACKED_WEIGHTS = 0x4
DTYPE_CODES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
NORM_MAX_H = 16384
NORM_CODES = {float("inf"): 0, 1.0: 1, 2.0: 2}


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} returned {STATUS_NAMES.get(status, status)}")


class Shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int64), ("I", ctypes.c_int64),
                ("E", ctypes.c_int64), ("k", ctypes.c_int32), ("flags", ctypes.c_int32)]


class RouterCfg(ctypes.Structure):
    _fields_ = [("score_fn", ctypes.c_int32), ("normalize", ctypes.c_int32),
                ("scale", ctypes.c_float), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("group_topn", ctypes.c_int32)]


class RouteShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("E", ctypes.c_int64), ("S", ctypes.c_int64), ("ld", ctypes.c_int64),
                ("k", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class NormShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int64), ("ld_x", ctypes.c_int64), ("ld_r", ctypes.c_int64),
                ("eps", ctypes.c_double), ("dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32)]


class GroupedShape(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int64), ("G", ctypes.c_int64), ("K", ctypes.c_int64), ("N", ctypes.c_int64),
                ("ld_x", ctypes.c_int64), ("ld_out", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_int32)]


class AdamWCfg(ctypes.Structure):
    _fields_ = [("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_float),
                ("weight_decay", ctypes.c_float), ("max_norm", ctypes.c_float), ("skip_nonfinite", ctypes.c_int32),
                ("missed", ctypes.c_void_p)]


class WsLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("err", "counts", "offsets", "mt_prefix", "perm_slot", "row_of", "meta", "router", "a",
                 "obuf", "combine", "dh", "aw", "dtw_part", "dlogits", "xp", "dyp", "dwr_part", "x_codes", "x_scales", "a_codes", "a_scales",
                 "mx_wgrad", "total")]


# name -> argument types (all return moe_status_t unless listed in _RESTYPES)
_P = ctypes.c_void_p
_SIG = {
    "moe_workspace_size": [ctypes.POINTER(Shape), ctypes.POINTER(ctypes.c_size_t)],
    "moe_workspace_layout": [ctypes.POINTER(Shape), ctypes.POINTER(WsLayout)],
    "moe_workspace_init": [_P, ctypes.c_size_t, _P],
    "moe_router": [_P, _P, _P, _P, ctypes.POINTER(Shape), ctypes.POINTER(RouterCfg), _P, _P, _P,
                   _P, ctypes.c_size_t, _P],
    "moe_router_noalloc": [_P, _P, _P, _P, ctypes.POINTER(Shape), ctypes.POINTER(RouterCfg), _P,
                           _P, _P, _P],
    "moe_router_noalloc_get_error": [ctypes.POINTER(ctypes.c_int32), _P],
    "moe_routing_metadata": [_P, ctypes.POINTER(Shape), _P, ctypes.c_size_t, _P],
    "moe_dispatch_gemm1": [_P, _P, ctypes.POINTER(Shape), _P, _P, ctypes.c_size_t, _P],
    "moe_swiglu_gemm2_combine": [_P, _P, _P, ctypes.POINTER(Shape), _P, _P, ctypes.c_size_t, _P],
    "moe_forward": [_P, _P, _P, _P, _P, ctypes.POINTER(Shape), _P, _P, ctypes.c_size_t, _P],
    "moe_route_logits": [_P, _P, _P, ctypes.POINTER(Shape), ctypes.POINTER(RouterCfg), _P, _P, _P, _P,
                         ctypes.c_size_t, _P],
    "moe_router_train": [_P, _P, _P, _P, ctypes.POINTER(Shape), ctypes.POINTER(RouterCfg), _P, _P,
                         _P, _P, _P, ctypes.c_size_t, _P],
    "moe_dispatch_gemm1_train": [_P, _P, ctypes.POINTER(Shape), _P, _P, _P, ctypes.c_size_t, _P],
    "moe_backward_stage2_data": [_P, _P, _P, _P, ctypes.POINTER(Shape), _P, _P, ctypes.c_size_t, _P],
    "moe_backward_stage2_weight": [_P, ctypes.POINTER(Shape), _P, _P, ctypes.c_size_t, _P],
    "moe_router_backward": [_P, _P, _P, _P, _P, ctypes.POINTER(Shape), ctypes.POINTER(RouterCfg), _P,
                            _P, ctypes.c_size_t, _P],
    "moe_backward_stage1_data": [_P, _P, _P, ctypes.POINTER(RouterCfg), ctypes.POINTER(Shape), _P, _P,
                                 ctypes.c_size_t, _P],
    "moe_backward_stage1_weight": [_P, ctypes.POINTER(Shape), _P, _P, ctypes.c_size_t, _P],
    "moe_backward": [_P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.POINTER(Shape),
                     ctypes.POINTER(RouterCfg), _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_mx_quantize": [_P, ctypes.c_int64, ctypes.c_int64, _P, _P, _P],
    "moe_mx_quantize_dispatch": [_P, ctypes.POINTER(Shape), _P, ctypes.c_size_t, _P],
    "moe_dispatch_gemm1_mx": [_P, _P, ctypes.POINTER(Shape), _P, _P, _P, ctypes.c_size_t, _P],
    "moe_dispatch_gemm1_mx_train": [_P, _P, ctypes.POINTER(Shape), _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_backward_stage2_weight_mx": [_P, ctypes.POINTER(Shape), _P, _P, ctypes.c_size_t, _P],
    "moe_backward_stage1_weight_mx": [_P, ctypes.POINTER(Shape), _P, _P, ctypes.c_size_t, _P],
    "moe_swiglu_gemm2_combine_mx": [_P, _P, _P, _P, _P, ctypes.POINTER(Shape), _P, _P, ctypes.c_size_t, _P],
    "moe_forward_mx": [_P, _P, _P, _P, _P, _P, _P, ctypes.POINTER(Shape), _P, _P, ctypes.c_size_t, _P],
    "moe_dispatch_rows": [_P, _P, ctypes.POINTER(Shape), _P, _P, _P, ctypes.c_size_t, _P],
    "moe_combine_rows": [_P, ctypes.POINTER(Shape), _P, _P, ctypes.c_size_t, _P],
    "moe_ep_pack": [_P, _P, ctypes.POINTER(Shape), ctypes.c_int32, ctypes.c_int64, _P, _P, _P, _P,
                    ctypes.c_size_t, _P],
    "moe_ep_receive_metadata": [_P, ctypes.c_int32, ctypes.c_int64, ctypes.POINTER(Shape), _P, ctypes.c_size_t,
                                _P],
    "moe_ep_combine": [_P, ctypes.POINTER(Shape), ctypes.c_int32, ctypes.c_int64, _P, _P, ctypes.c_size_t, _P],
    "moe_packed_weights_size": [ctypes.POINTER(Shape), ctypes.POINTER(ctypes.c_size_t),
                                ctypes.POINTER(ctypes.c_size_t)],
    "moe_pack_weights": [_P, _P, ctypes.POINTER(Shape), _P, _P, _P],
    "moe_route_workspace_size": [ctypes.POINTER(RouteShape), ctypes.POINTER(ctypes.c_size_t)],
    "moe_route": [_P, _P, _P, _P, ctypes.POINTER(RouteShape), ctypes.POINTER(RouterCfg), _P, _P, _P, _P, _P, _P,
                  ctypes.c_size_t, _P],
    "moe_route_backward": [_P, _P, _P, ctypes.POINTER(RouteShape), ctypes.POINTER(RouterCfg), _P, _P, _P, _P, _P, _P,
                           _P],
    "moe_bias_update": [_P, _P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_float, _P],
    "moe_tensors_workspace_size": [ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)],
    "moe_grad_norm": [_P, _P, _P, ctypes.c_int32, ctypes.c_int32, _P, _P, ctypes.c_size_t, _P],
    "moe_clip_grads": [_P, _P, _P, ctypes.c_int32, ctypes.c_int32, ctypes.c_float, _P, _P, ctypes.c_size_t, _P],
    "moe_adamw": [_P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int32, ctypes.POINTER(AdamWCfg), _P, _P, _P, _P,
                  ctypes.c_size_t, _P],
    "moe_mx_dispatch": [_P, _P, ctypes.POINTER(Shape), _P, ctypes.c_size_t, _P],
    "moe_forward_mx_codes": [_P, _P, _P, _P, _P, _P, _P, _P, ctypes.POINTER(Shape), _P, _P, ctypes.c_size_t, _P],
    "moe_rms_norm": [_P, _P, _P, ctypes.POINTER(NormShape), _P, _P, _P, _P, _P, _P],
    "moe_rms_norm_workspace_size": [ctypes.c_int64, ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)],
    "moe_rms_norm_backward": [_P, _P, _P, _P, _P, ctypes.POINTER(NormShape), _P, _P, _P, ctypes.c_size_t, _P],
    "moe_grouped_workspace_size": [ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)],
    "moe_grouped_mm": [_P, _P, _P, ctypes.POINTER(GroupedShape), _P, _P, ctypes.c_size_t, _P],
    "moe_grouped_wgrad": [_P, _P, _P, ctypes.POINTER(GroupedShape), _P, _P, ctypes.c_size_t, _P],
    "moe_grouped_mm_mx": [_P, _P, _P, _P, _P, ctypes.POINTER(GroupedShape), _P, _P, ctypes.c_size_t, _P],
    "moe_get_device_error": [_P, ctypes.POINTER(ctypes.c_int32), _P],
    "moe_status_string": [ctypes.c_int],
    "moe_kernel_launch_count": [],
}
_RESTYPES = {"moe_status_string": ctypes.c_char_p, "moe_kernel_launch_count": ctypes.c_uint64}

_lib = None
_native = None


def load(path: str = LIB_PATH):
    """Load libmoe.so (built by moe_expert_router_gb300.build); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    for name, args in _SIG.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = _RESTYPES.get(name, ctypes.c_int)
    _lib = lib
    return lib


def _check(fn: str, status: int):
    if status != MOE_OK:
        raise MoEError(fn, status)


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch tensor")
    if not t.is_cuda:
        raise ValueError("libmoe takes CUDA tensors only")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream, like):
    if stream is None:
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(like.get_device()))
    return ctypes.c_void_p(stream.cuda_stream)


def shape(T, H, I, E, k, training=False, mxfp8=False, packed=False) -> Shape:
    flags = ((SHAPE_TRAINING if training else 0) | (SHAPE_MXFP8 if mxfp8 else 0) |
             (SHAPE_PACKED_WEIGHTS if packed else 0))
    return Shape(int(T), int(H), int(I), int(E), int(k), flags)


def router_cfg(score="softmax", normalize=True, scale=1.0, n_group=1, topk_group=1,
               group_topn=2) -> RouterCfg:
    fn = SCORE_SOFTMAX if score == "softmax" else SCORE_SIGMOID
    return RouterCfg(fn, int(bool(normalize)), float(scale), int(n_group), int(topk_group),
                     int(group_topn))


def moe_workspace_size(shp: Shape) -> int:
    n = ctypes.c_size_t()
    _check("moe_workspace_size", load().moe_workspace_size(ctypes.byref(shp), ctypes.byref(n)))
    return int(n.value)


def moe_workspace_layout(shp: Shape) -> WsLayout:
    L = WsLayout()
    _check("moe_workspace_layout", load().moe_workspace_layout(ctypes.byref(shp), ctypes.byref(L)))
    return L


def moe_workspace_init(ws, stream=None):
    _check("moe_workspace_init",
           load().moe_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream, ws)))


def moe_router(x, w_r, shp, cfg, topk_idx, topk_w, ws, aux=None, logit_offset=None,
               sel_bias=None, stream=None):
    _check("moe_router", load().moe_router(
        _ptr(x), _ptr(w_r), _ptr(logit_offset), _ptr(sel_bias), ctypes.byref(shp),
        ctypes.byref(cfg), _ptr(topk_idx), _ptr(topk_w), _ptr(aux), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream, x)))


def moe_router_noalloc(x, w_r, shp, cfg, topk_idx, topk_w, aux=None, logit_offset=None,
                       sel_bias=None, stream=None):
    """moe_router without a workspace: for callers that may not allocate device
    memory (the scratch lives in a static array inside libmoe; T * E <= 2**20, E * H <= 2**20)."""
    _check("moe_router_noalloc", load().moe_router_noalloc(
        _ptr(x), _ptr(w_r), _ptr(logit_offset), _ptr(sel_bias), ctypes.byref(shp),
        ctypes.byref(cfg), _ptr(topk_idx), _ptr(topk_w), _ptr(aux), _stream(stream, x)))


def moe_router_noalloc_get_error(stream=None) -> int:
    """Wait for the stream, return and clear moe_router_noalloc's error word on
    the current device (0 = none)."""
    import torch
    code = ctypes.c_int32()
    if stream is None:
        stream = torch.cuda.current_stream()
    st = load().moe_router_noalloc_get_error(ctypes.byref(code), ctypes.c_void_p(stream.cuda_stream))
    if st not in (MOE_OK, 5):
        raise MoEError("moe_router_noalloc_get_error", st)
    return int(code.value)


def moe_routing_metadata(topk_idx, shp, ws, stream=None):
    _check("moe_routing_metadata", load().moe_routing_metadata(
        _ptr(topk_idx), ctypes.byref(shp), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream, topk_idx)))


def moe_dispatch_gemm1(x, w1, shp, a, ws, stream=None):
    _check("moe_dispatch_gemm1", load().moe_dispatch_gemm1(
        _ptr(x), _ptr(w1), ctypes.byref(shp), _ptr(a), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream, x)))


def moe_swiglu_gemm2_combine(a, topk_w, w2, shp, y, ws, stream=None):
    _check("moe_swiglu_gemm2_combine", load().moe_swiglu_gemm2_combine(
        _ptr(a), _ptr(topk_w), _ptr(w2), ctypes.byref(shp), _ptr(y), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream, a)))


def moe_forward(x, topk_idx, topk_w, w1, w2, shp, y, ws, stream=None):
    _check("moe_forward", load().moe_forward(
        _ptr(x), _ptr(topk_idx), _ptr(topk_w), _ptr(w1), _ptr(w2), ctypes.byref(shp), _ptr(y),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream, x)))


def _cfg_ref(cfg):
    return None if cfg is None else ctypes.byref(cfg)


def _nbytes(ws):
    return ws.numel() * ws.element_size()


def moe_route_logits(logits, shp, cfg, topk_idx, topk_w, ws, aux=None, logit_offset=None,
                     sel_bias=None, stream=None):
    """Routing from given fp32 logits [T, E] (random logits: the `uniform` force-balance mode)."""
    _check("moe_route_logits", load().moe_route_logits(
        _ptr(logits), _ptr(logit_offset), _ptr(sel_bias), ctypes.byref(shp), ctypes.byref(cfg),
        _ptr(topk_idx), _ptr(topk_w), _ptr(aux), _ptr(ws), _nbytes(ws), _stream(stream, logits)))


def moe_router_train(x, w_r, shp, cfg, topk_idx, topk_w, logits, ws, aux=None, logit_offset=None,
                     sel_bias=None, stream=None):
    """moe_router that also writes the fp32 logits [T, E] for moe_router_backward."""
    _check("moe_router_train", load().moe_router_train(
        _ptr(x), _ptr(w_r), _ptr(logit_offset), _ptr(sel_bias), ctypes.byref(shp),
        ctypes.byref(cfg), _ptr(topk_idx), _ptr(topk_w), _ptr(aux), _ptr(logits), _ptr(ws),
        _nbytes(ws), _stream(stream, x)))


def moe_dispatch_gemm1_train(x, w1, shp, a, h, ws, stream=None):
    """moe_dispatch_gemm1 that also stores the pre-activation h [T*k, 2I] (routed order)."""
    _check("moe_dispatch_gemm1_train", load().moe_dispatch_gemm1_train(
        _ptr(x), _ptr(w1), ctypes.byref(shp), _ptr(a), _ptr(h), _ptr(ws), _nbytes(ws),
        _stream(stream, x)))


def moe_backward_stage2_data(dy, topk_w, w2, h, shp, ws, dtopk_w=None, stream=None):
    _check("moe_backward_stage2_data", load().moe_backward_stage2_data(
        _ptr(dy), _ptr(topk_w), _ptr(w2), _ptr(h), ctypes.byref(shp), _ptr(dtopk_w), _ptr(ws),
        _nbytes(ws), _stream(stream, ws)))


def moe_backward_stage2_weight(dy, shp, dw2, ws, stream=None):
    _check("moe_backward_stage2_weight", load().moe_backward_stage2_weight(
        _ptr(dy), ctypes.byref(shp), _ptr(dw2), _ptr(ws), _nbytes(ws), _stream(stream, ws)))


def moe_router_backward(x, logits, topk_idx, topk_w, dtopk_w, shp, cfg, dw_r, ws, stream=None):
    _check("moe_router_backward", load().moe_router_backward(
        _ptr(x), _ptr(logits), _ptr(topk_idx), _ptr(topk_w), _ptr(dtopk_w), ctypes.byref(shp),
        ctypes.byref(cfg), _ptr(dw_r), _ptr(ws), _nbytes(ws), _stream(stream, ws)))


def moe_backward_stage1_data(w1, shp, dx, ws, w_r=None, topk_idx=None, cfg=None, stream=None):
    _check("moe_backward_stage1_data", load().moe_backward_stage1_data(
        _ptr(w1), _ptr(w_r), _ptr(topk_idx), _cfg_ref(cfg), ctypes.byref(shp), _ptr(dx), _ptr(ws),
        _nbytes(ws), _stream(stream, ws)))


def moe_backward_stage1_weight(x, shp, dw1, ws, stream=None):
    _check("moe_backward_stage1_weight", load().moe_backward_stage1_weight(
        _ptr(x), ctypes.byref(shp), _ptr(dw1), _ptr(ws), _nbytes(ws), _stream(stream, ws)))


def moe_backward(x, topk_idx, topk_w, w1, w2, h, dy, shp, dx, dw1, dw2, ws, w_r=None, logits=None,
                 cfg=None, dw_r=None, dtopk_w=None, stream=None):
    _check("moe_backward", load().moe_backward(
        _ptr(x), _ptr(w_r), _ptr(logits), _ptr(topk_idx), _ptr(topk_w), _ptr(w1), _ptr(w2), _ptr(h),
        _ptr(dy), ctypes.byref(shp), _cfg_ref(cfg), _ptr(dx), _ptr(dw1), _ptr(dw2), _ptr(dw_r),
        _ptr(dtopk_w), _ptr(ws), _nbytes(ws), _stream(stream, ws)))


def mx_scales_empty(shape, device):
    """An uninitialised buffer for the k-block-major E8M0 scales of an MXFP8
    tensor of `shape` (rows = the product of the leading dimensions, cols the
    last, a multiple of 128): uint8 [cols / 128, *shape[:-1], 4] when rows is a
    multiple of 4, else [cols / 128, rows rounded up to 4, 4] -- one 32-bit word
    per row and 128-column block, rows consecutive within a block."""
    shape = tuple(shape)
    rows = 1
    for d in shape[:-1]:
        rows *= d
    lead = shape[:-1] if rows % 4 == 0 else ((rows + 3) // 4 * 4,)
    return torch.empty((shape[-1] // 128,) + lead + (4,), dtype=torch.uint8, device=device)


def moe_mx_quantize(t, codes, scales, stream=None):
    """MXFP8 quantization of a bf16 tensor along its last dimension (a multiple of
    128): codes uint8 of the same shape, scales k-block-major (``mx_scales_empty``)."""
    cols = t.shape[-1]
    rows = t.numel() // cols if cols else 0
    if codes.numel() != t.numel() or scales.numel() * 32 != (rows + 3) // 4 * 4 * cols:
        raise ValueError("codes must match t and scales hold the k-block-major words of rows rounded up to 4")
    _check("moe_mx_quantize", load().moe_mx_quantize(_ptr(t), rows, cols, _ptr(codes), _ptr(scales),
                                                     _stream(stream, t)))


def moe_mx_quantize_dispatch(x, shp, ws, stream=None):
    """The MXFP8 dispatch: x quantized into the workspace in routed-row order."""
    _check("moe_mx_quantize_dispatch", load().moe_mx_quantize_dispatch(
        _ptr(x), ctypes.byref(shp), _ptr(ws), _nbytes(ws), _stream(stream, ws)))


def moe_dispatch_gemm1_mx(w1q, w1s, shp, aq, as_, ws, stream=None):
    _check("moe_dispatch_gemm1_mx", load().moe_dispatch_gemm1_mx(
        _ptr(w1q), _ptr(w1s), ctypes.byref(shp), _ptr(aq), _ptr(as_), _ptr(ws), _nbytes(ws),
        _stream(stream, ws)))


def moe_dispatch_gemm1_mx_train(w1q, w1s, shp, aq, as_, h, ws, stream=None):
    _check("moe_dispatch_gemm1_mx_train", load().moe_dispatch_gemm1_mx_train(
        _ptr(w1q), _ptr(w1s), ctypes.byref(shp), _ptr(aq), _ptr(as_), _ptr(h), _ptr(ws), _nbytes(ws),
        _stream(stream, ws)))


def moe_backward_stage2_weight_mx(dy, shp, dw2, ws, stream=None):
    _check("moe_backward_stage2_weight_mx", load().moe_backward_stage2_weight_mx(
        _ptr(dy), ctypes.byref(shp), _ptr(dw2), _ptr(ws), _nbytes(ws), _stream(stream, ws)))


def moe_backward_stage1_weight_mx(x, shp, dw1, ws, stream=None):
    _check("moe_backward_stage1_weight_mx", load().moe_backward_stage1_weight_mx(
        _ptr(x), ctypes.byref(shp), _ptr(dw1), _ptr(ws), _nbytes(ws), _stream(stream, ws)))


def moe_swiglu_gemm2_combine_mx(aq, as_, topk_w, w2q, w2s, shp, y, ws, stream=None):
    _check("moe_swiglu_gemm2_combine_mx", load().moe_swiglu_gemm2_combine_mx(
        _ptr(aq), _ptr(as_), _ptr(topk_w), _ptr(w2q), _ptr(w2s), ctypes.byref(shp), _ptr(y), _ptr(ws),
        _nbytes(ws), _stream(stream, ws)))


def moe_forward_mx(x, topk_idx, topk_w, w1q, w1s, w2q, w2s, shp, y, ws, stream=None):
    _check("moe_forward_mx", load().moe_forward_mx(
        _ptr(x), _ptr(topk_idx), _ptr(topk_w), _ptr(w1q), _ptr(w1s), _ptr(w2q), _ptr(w2s),
        ctypes.byref(shp), _ptr(y), _ptr(ws), _nbytes(ws), _stream(stream, ws)))


def moe_mx_dispatch(x_codes, x_scales, shp, ws, stream=None):
    """The MXFP8 dispatch of tokens that are quantized already (moe_rms_norm's codes and scales)."""
    _check("moe_mx_dispatch", load().moe_mx_dispatch(
        _ptr(x_codes), _ptr(x_scales), ctypes.byref(shp), _ptr(ws), _nbytes(ws), _stream(stream, ws)))


def moe_forward_mx_codes(x_codes, x_scales, topk_idx, topk_w, w1q, w1s, w2q, w2s, shp, y, ws, stream=None):
    """moe_forward_mx from tokens that are quantized already."""
    _check("moe_forward_mx_codes", load().moe_forward_mx_codes(
        _ptr(x_codes), _ptr(x_scales), _ptr(topk_idx), _ptr(topk_w), _ptr(w1q), _ptr(w1s), _ptr(w2q), _ptr(w2s),
        ctypes.byref(shp), _ptr(y), _ptr(ws), _nbytes(ws), _stream(stream, ws)))


def moe_dispatch_rows(x, shp, rows, ws, topk_w=None, row_weight=None, stream=None):
    """rows[r] = x[token of routed row r] (and row_weight[r] = its routing weight): the
    send buffer of an expert-parallel dispatch."""
    _check("moe_dispatch_rows", load().moe_dispatch_rows(
        _ptr(x), _ptr(topk_w), ctypes.byref(shp), _ptr(rows), _ptr(row_weight), _ptr(ws), _nbytes(ws),
        _stream(stream, ws)))


def moe_ep_pack(x, topk_w, shp, n_ranks, capacity, send_rows, send_w, send_counts, ws, stream=None):
    """Expert parallelism, sender: fixed-size send blocks of capacity rows per rank."""
    _check("moe_ep_pack", load().moe_ep_pack(
        _ptr(x), _ptr(topk_w), ctypes.byref(shp), int(n_ranks), int(capacity), _ptr(send_rows), _ptr(send_w),
        _ptr(send_counts), _ptr(ws), _nbytes(ws), _stream(stream, ws)))


def moe_ep_receive_metadata(recv_counts, n_ranks, capacity, recv_shp, ws, stream=None):
    """Expert parallelism, receiver: routing metadata of the received blocks from their counts."""
    _check("moe_ep_receive_metadata", load().moe_ep_receive_metadata(
        _ptr(recv_counts), int(n_ranks), int(capacity), ctypes.byref(recv_shp), _ptr(ws), _nbytes(ws),
        _stream(stream, ws)))


def moe_ep_combine(back_rows, shp, n_ranks, capacity, y, ws, stream=None):
    """Expert parallelism, sender: the sum of each token's returned rows."""
    _check("moe_ep_combine", load().moe_ep_combine(
        _ptr(back_rows), ctypes.byref(shp), int(n_ranks), int(capacity), _ptr(y), _ptr(ws), _nbytes(ws),
        _stream(stream, ws)))


def moe_combine_rows(rows, shp, y, ws, stream=None):
    """y[t] = sum of the token's (already weighted) rows, in routed order."""
    _check("moe_combine_rows", load().moe_combine_rows(
        _ptr(rows), ctypes.byref(shp), _ptr(y), _ptr(ws), _nbytes(ws), _stream(stream, ws)))


def moe_get_device_error(ws, stream=None) -> int:
    """Wait for the stream, return and clear the workspace error word (0 = none)."""
    code = ctypes.c_int32()
    st = load().moe_get_device_error(_ptr(ws), ctypes.byref(code), _stream(stream, ws))
    if st not in (MOE_OK, 5):
        raise MoEError("moe_get_device_error", st)
    return int(code.value)


def moe_kernel_launch_count() -> int:
    return int(load().moe_kernel_launch_count())


def moe_packed_weights_size(shp: Shape) -> tuple:
    """Bytes of the tile-packed w1 and w2 for this shape."""
    a, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check("moe_packed_weights_size", load().moe_packed_weights_size(ctypes.byref(shp), ctypes.byref(a),
                                                                     ctypes.byref(b)))
    return a.value, b.value


def moe_pack_weights(w1, w2, shp: Shape, w1p=None, w2p=None, stream=None):
    """Tile-packed copies of w1 [E, 2I, H] and w2 [E, H, I] (uint8 tensors, allocated when
    not given; either weight may be None to skip it). Pass them to the forward calls with a
    shape made with packed=True."""
    n1, n2 = moe_packed_weights_size(shp)
    like = w1 if w1 is not None else w2
    if w1 is not None and w1p is None:
        w1p = torch.empty(n1, dtype=torch.uint8, device=like.device)
    if w2 is not None and w2p is None:
        w2p = torch.empty(n2, dtype=torch.uint8, device=like.device)
    _check("moe_pack_weights", load().moe_pack_weights(
        _ptr(w1) if w1 is not None else None, _ptr(w2) if w2 is not None else None, ctypes.byref(shp),
        _ptr(w1p) if w1 is not None else None, _ptr(w2p) if w2 is not None else None, _stream(stream, like)))
    return w1p, w2p


def new_workspace(shp: Shape, device=None) -> torch.Tensor:
    """A 256-byte aligned uint8 workspace of the required size, header zeroed."""
    n = moe_workspace_size(shp)
    ws = torch.empty(n + 256, dtype=torch.uint8, device=device or "cuda")
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + n]
    moe_workspace_init(ws)
    return ws


# ------------------------------------------------------------------ the trainable router

def _module():
    """csrc/native.cpp, bound to the library: the calls whose cost on the host shows."""
    global _native
    if _native is None:
        lib = load()
        try:
            from . import _native as native
        except ImportError as e:
            raise RuntimeError(f"{NATIVE_PATH} is missing: build it first "
                               "(python -c 'import __graft_entry__ as g; g.build()')") from e
        native.bind(*[ctypes.cast(f, ctypes.c_void_p).value for f in
                      (lib.moe_route, lib.moe_route_backward, lib.moe_bias_update, lib.moe_grad_norm,
                       lib.moe_clip_grads, lib.moe_adamw, lib.moe_grouped_mm, lib.moe_grouped_wgrad,
                       lib.moe_grouped_mm_mx, lib.moe_rms_norm, lib.moe_rms_norm_backward)])
        _native = native
    return _native


def _raw_stream(stream, like):
    """A stream's handle as a number; the current one's of the tensor's device for None."""
    if stream is not None:
        return stream.cuda_stream
    try:
        device = like.get_device()
    except AttributeError:
        raise TypeError(f"expected a torch tensor, not {type(like).__name__}") from None
    return torch._C._cuda_getCurrentRawStream(device) if device >= 0 else 0


@functools.lru_cache(maxsize=256)
def moe_route_workspace_size(T, E, S=1, k=1) -> int:
    n = ctypes.c_size_t()
    shp = RouteShape(T, E, S, E, k, 0)
    _check("moe_route_workspace_size", load().moe_route_workspace_size(ctypes.byref(shp), ctypes.byref(n)))
    return int(n.value)


def moe_route(logits, cfg, topk_idx, topk_w, sel_bias=None, token_mask=None, seq_offsets=None, counts=None,
              seq_tokens=None, losses=None, ws=None, stream=None):
    """Selection from logits [T, E] (fp32, bf16 or fp16; rows may be apart), with the balance
    statistics of a training step where counts [S, E], seq_tokens [S + 2], losses [2] and a
    workspace of moe_route_workspace_size bytes are given. token_mask: bool or uint8 [T]."""
    _check("moe_route", _module().route(logits, ctypes.addressof(cfg), topk_idx, topk_w, sel_bias, token_mask, seq_offsets,
                                        counts, seq_tokens, losses, ws, _raw_stream(stream, logits)))


def moe_route_backward(logits, cfg, topk_idx, dtopk_w, dlogits, token_mask=None, seq_offsets=None, counts=None,
                       seq_tokens=None, dlosses=None, stream=None):
    """Gradient of moe_route's topk_w and losses with respect to the logits, into dlogits [T, E]
    (dense, the logits' type)."""
    _check("moe_route_backward", _module().route_backward(
        logits, ctypes.addressof(cfg), topk_idx, dtopk_w, dlogits, token_mask, seq_offsets, counts, seq_tokens, dlosses,
        _raw_stream(stream, logits)))


def moe_bias_update(bias, counts, rate, stream=None):
    """bias [E] or [L, E] += rate * sign(mean count - count), in place; counts int32 [S, E] or
    [L, S, E], added over the sequences."""
    _check("moe_bias_update", _module().bias_update(bias, counts, float(rate), _raw_stream(stream, bias)))


# ------------------------------------------------------------------ the norm in front of the layer

def moe_rms_norm(x, weight, y, eps=1e-6, residual=None, h=None, rstd=None, codes=None, scales=None, stream=None):
    """y = the root-mean-square norm of h = x + residual (of x without one), times weight; x [T, H]
    fp32, bf16 or fp16 (rows of x and residual may be apart). h (the stream, which may be x's or
    residual's own memory), rstd fp32 [T] (for the backward) and codes uint8 [T, H] with scales
    (``mx_scales_empty((T, H))``: y in MXFP8, H a multiple of 128) are written where given; y may be
    None beside codes."""
    _check("moe_rms_norm", _module().rms_norm(x, weight, y, eps, residual, h, rstd, codes, scales, _raw_stream(stream, x)))


@functools.lru_cache(maxsize=256)
def moe_rms_norm_workspace_size(T, H) -> int:
    n = ctypes.c_size_t()
    _check("moe_rms_norm_workspace_size", load().moe_rms_norm_workspace_size(T, H, ctypes.byref(n)))
    return int(n.value)


def rms_norm_scratch(T, H, like) -> torch.Tensor:
    """A workspace for the backward of T rows of H on the device of `like`."""
    return torch.empty(moe_rms_norm_workspace_size(T, H), dtype=torch.uint8, device=like.device)


def moe_rms_norm_backward(dy, h, weight, rstd, dx, dweight, ws, dh=None, stream=None):
    """dx (of x and of residual) and dweight of moe_rms_norm, from dy and, where the stream h went on
    by itself, its gradient dh."""
    _check("moe_rms_norm_backward", _module().rms_norm_backward(dy, h, weight, rstd, dx, dweight, ws, dh,
                                                                _raw_stream(stream, h)))


# ------------------------------------------------------------------ products grouped by expert

@functools.lru_cache(maxsize=256)
def moe_grouped_workspace_size(G) -> int:
    n = ctypes.c_size_t()
    _check("moe_grouped_workspace_size", load().moe_grouped_workspace_size(G, ctypes.byref(n)))
    return int(n.value)


def grouped_workspace(G, device=None) -> torch.Tensor:
    """A workspace for the products of up to G groups, its header zeroed. Calls that share one are
    ordered on one stream."""
    ws = torch.empty(moe_grouped_workspace_size(G), dtype=torch.uint8, device=device or "cuda")
    moe_workspace_init(ws)
    return ws


def moe_grouped_mm(x, w, offsets, out, ws, transposed=False, stream=None, nan_on_bad=False):
    """out[r] = x[r] . w[g]^T for the rows offsets[g] .. offsets[g + 1] - 1 of each group g; x [R, K]
    and out [R, N] bf16 or fp16 (rows may be apart), w [G, N, K], or with transposed w [G, K, N] and
    out[r] = x[r] . w[g]; offsets int32 [G + 1] on the device. Rows of no group are left alone. Offsets that
    decrease or leave [0, R] set DEVERR_BAD_OFFSETS in ws and leave out alone, or with nan_on_bad fill it with
    NaN."""
    _check("moe_grouped_mm", _module().grouped_mm(x, w, offsets, out, ws, bool(transposed), bool(nan_on_bad),
                                                  _raw_stream(stream, x)))


def moe_grouped_wgrad(a, b, offsets, dw, ws, stream=None, nan_on_bad=False):
    """dw[g] = the sum over group g's rows of a[r]^T b[r]; a [R, N], b [R, K], dw [G, N, K] of one type. Of bad
    offsets dw is 0, or with nan_on_bad NaN."""
    _check("moe_grouped_wgrad", _module().grouped_wgrad(a, b, offsets, dw, ws, bool(nan_on_bad), _raw_stream(stream, a)))


def moe_grouped_mm_mx(x_codes, x_scales, w_codes, w_scales, offsets, out, ws, stream=None):
    """moe_grouped_mm on MXFP8 operands (moe_mx_quantize's format): x [R, K], w [G, N, K], out bf16 [R, N]."""
    _check("moe_grouped_mm_mx", _module().grouped_mm_mx(x_codes, x_scales, w_codes, w_scales, offsets, out, ws,
                                                        _raw_stream(stream, x_codes)))


# ------------------------------------------------------------------ lists of tensors

@functools.lru_cache(maxsize=256)
def moe_tensors_workspace_size(n) -> int:
    size = ctypes.c_size_t()
    _check("moe_tensors_workspace_size", load().moe_tensors_workspace_size(n, ctypes.byref(size)))
    return int(size.value)


def tensors_scratch(n, like):
    """A workspace for lists of n tensors on the device of `like`, and a scalar for their norm."""
    return _module().scratch(moe_tensors_workspace_size(n), like)


def _norm_code(norm_type):
    try:
        return NORM_CODES[float(norm_type)]
    except KeyError:
        raise ValueError(f"norm_type must be 1, 2 or inf, not {norm_type}") from None


def moe_grad_norm(grads, norm, ws, norm_type=2.0, stream=None):
    """norm (one fp32 element) = the norm of all the tensors' elements together."""
    _check("moe_grad_norm", _module().grad_norm(grads, _norm_code(norm_type), norm, ws, _raw_stream(stream, norm)))


def moe_clip_grads(grads, max_norm, norm, ws, norm_type=2.0, stream=None):
    """The same norm, and every tensor times min(1, max_norm / (norm + 1e-6)), in place."""
    _check("moe_clip_grads", _module().clip_grads(grads, _norm_code(norm_type), float(max_norm), norm, ws,
                                                  _raw_stream(stream, norm)))


def moe_adamw(params, grads, exp_avg, exp_avg_sq, lr, step, ws, cfg, masters=None, norm=None, stream=None,
              missed=None):
    """One AdamW step over lists of tensors, in place; masters: a list with an fp32 tensor or None
    for each parameter, or None; missed: int32, the steps that each parameter had no part in, or
    None (it takes the place of cfg.missed)."""
    _check("moe_adamw", _module().adamw(params, grads, exp_avg, exp_avg_sq, masters, ctypes.addressof(cfg), lr, step, norm,
                                        ws, missed, _raw_stream(stream, lr)))
