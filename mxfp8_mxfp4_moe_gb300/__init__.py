"""Python binding of libkmoe: the Kimi-K3 routed-expert MoE forward
(MXFP8 activations x MXFP4 weights, SiTU) for GB300 (sm_103a).

Argument marshalling only: every step runs in the library's CUDA kernels.
The functions carry the C entry points' names (include/kmoe.h); torch is used
for device memory and the current stream.  Tensors live on the current GPU.
With `stream` a call runs on that stream and allocates from its memory; the
caller orders it with the streams that make and use the tensors.  Importing
this package loads the in-tree libkmoe.so and raises if it is missing (build it with
`python -m mxfp8_mxfp4_moe_gb300.build` or __graft_entry__.build()).
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkmoe.so")

KMOE_OK = 0
STATUS = {0: "KMOE_OK", 1: "KMOE_ERR_ARG", 2: "KMOE_ERR_SHAPE", 3: "KMOE_ERR_ALIGN", 4: "KMOE_ERR_ARCH",
          5: "KMOE_ERR_WORKSPACE", 6: "KMOE_ERR_CUDA", 7: "KMOE_ERR_TIMEOUT", 8: "KMOE_ERR_DEVICE"}
KMOE_MXFP8_E4M3 = 0
KMOE_MXFP4_E2M1 = 1

EXPORTS = ("kmoe_status_string", "kmoe_check_device", "kmoe_workspace_size", "kmoe_workspace_layout",
           "kmoe_route", "kmoe_quantize_mx", "kmoe_prepared_weight_bytes", "kmoe_prepare_weights",
           "kmoe_forward", "kmoe_forward_ex", "kmoe_device_error", "kmoe_tile_sf_offset",
           "kmoe_selftest_wait_timeout", "kmoe_forward_noalloc", "kmoe_mma_peak_run",
           "kmoe_router_workspace_size", "kmoe_router", "kmoe_forward_router", "kmoe_selftest_activation",
           "kmoe_rmsnorm", "kmoe_rmsnorm_workspace_size", "kmoe_rmsnorm_backward", "kmoe_route_grouped",
           "kmoe_route_backward", "kmoe_combine_backward", "kmoe_forward_mx")
NOALLOC_SCRATCH_BYTES = 32 << 20


class kmoe_params(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("H", ctypes.c_int), ("I", ctypes.c_int), ("E", ctypes.c_int),
                ("k", ctypes.c_int), ("situ_beta", ctypes.c_float), ("situ_linear_beta", ctypes.c_float),
                ("routed_scaling_factor", ctypes.c_float), ("flags", ctypes.c_uint32),
                ("swiglu_alpha", ctypes.c_float), ("swiglu_beta", ctypes.c_float), ("swiglu_limit", ctypes.c_float)]


class kmoe_ws_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("err", "topk_ids", "topk_w", "counts", "seg_start", "tile_start",
                                               "row_of_slot", "slot_of_row", "xq", "xsf", "iq", "isf", "y")] + \
               [("tile_rows", ctypes.c_int), ("max_tiles", ctypes.c_int), ("total", ctypes.c_size_t),
                ("logits", ctypes.c_size_t), ("tile_start_big", ctypes.c_size_t), ("xsf_big", ctypes.c_size_t),
                ("isf_big", ctypes.c_size_t), ("tile_rows_big", ctypes.c_int), ("max_tiles_big", ctypes.c_int),
                ("big_rows", ctypes.c_int)]


class kmoe_route_params(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("E", ctypes.c_int), ("k", ctypes.c_int), ("n_group", ctypes.c_int),
                ("topk_group", ctypes.c_int), ("flags", ctypes.c_uint32), ("scale", ctypes.c_float)]


class kmoe_stage_events(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("start", "routed", "permuted", "quantized", "fc1", "fc2",
                                               "combined")]


STAGE_NAMES = ("route", "permute", "quantize", "fc1", "fc2", "combine")


class KmoeError(RuntimeError):
    def __init__(self, fn, status, lib=None):
        msg = STATUS.get(status, str(status))
        if lib is not None:
            msg += ": " + lib.kmoe_status_string(status).decode()
        super().__init__(f"{fn} failed with {msg}")
        self.status = status


def load_library(path: str = LIB_PATH):
    if not os.path.exists(path):
        raise ImportError(f"libkmoe.so not built at {path}; run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    P, S, I, V = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_void_p
    pp = ctypes.POINTER(kmoe_params)
    lib.kmoe_status_string.restype = ctypes.c_char_p
    lib.kmoe_status_string.argtypes = [I]
    lib.kmoe_check_device.argtypes = [I]
    lib.kmoe_workspace_size.restype = S
    lib.kmoe_workspace_size.argtypes = [pp]
    lib.kmoe_workspace_layout.argtypes = [pp, ctypes.POINTER(kmoe_ws_layout)]
    lib.kmoe_route.argtypes = [P, P, I, I, I, P, P, V]
    lib.kmoe_quantize_mx.argtypes = [P, I, I, I, P, P, V]
    lib.kmoe_prepared_weight_bytes.restype = S
    lib.kmoe_prepared_weight_bytes.argtypes = [pp, I]
    lib.kmoe_prepare_weights.argtypes = [pp, P, P, P, P, P, P, V]
    lib.kmoe_forward.argtypes = [pp, P, P, P, P, P, P, P, P, P, S, V]
    lib.kmoe_forward_ex.argtypes = [pp, P, P, P, P, P, P, P, P, P, S, V, ctypes.POINTER(kmoe_stage_events)]
    lib.kmoe_device_error.argtypes = [P, ctypes.POINTER(ctypes.c_uint32), V]
    lib.kmoe_tile_sf_offset.restype = S
    lib.kmoe_tile_sf_offset.argtypes = [I, I, I, I, I, I]
    lib.kmoe_selftest_wait_timeout.argtypes = [P, I, V]
    lib.kmoe_mma_peak_run.argtypes = [I, I, P, V]
    lib.kmoe_mma_peak_run.restype = ctypes.c_int
    lib.kmoe_forward_noalloc.argtypes = [pp, P, P, P, P, P, P, P, P, P, V]
    lib.kmoe_forward_noalloc.restype = ctypes.c_int
    lib.kmoe_router_workspace_size.restype = S
    lib.kmoe_router_workspace_size.argtypes = [I, I, I]
    lib.kmoe_router.argtypes = [P, P, P, I, I, I, I, P, P, P, P, S, V]
    lib.kmoe_forward_router.argtypes = [pp, P, P, P, P, P, P, P, S, V, ctypes.POINTER(kmoe_stage_events)]
    lib.kmoe_selftest_activation.argtypes = [pp, P, P, I, P, V]
    F, U = ctypes.c_float, ctypes.c_uint32
    rp = ctypes.POINTER(kmoe_route_params)
    lib.kmoe_rmsnorm.argtypes = [P, P, P, I, I, F, U, P, P, P, P, V]
    lib.kmoe_rmsnorm_workspace_size.restype = S
    lib.kmoe_rmsnorm_workspace_size.argtypes = [I, I]
    lib.kmoe_rmsnorm_backward.argtypes = [P, P, P, P, I, I, F, U, P, P, P, S, V]
    lib.kmoe_route_grouped.argtypes = [rp, P, P, P, P, V]
    lib.kmoe_route_backward.argtypes = [rp, P, P, P, P, V]
    lib.kmoe_combine_backward.argtypes = [P, P, P, I, I, I, I, F, P, V]
    lib.kmoe_forward_mx.argtypes = [pp, P, P, P, P, P, P, P, P, S, V]
    for n in ("kmoe_rmsnorm", "kmoe_rmsnorm_backward", "kmoe_route_grouped", "kmoe_route_backward",
              "kmoe_combine_backward", "kmoe_forward_mx"):
        getattr(lib, n).restype = ctypes.c_int
    for n in ("kmoe_check_device", "kmoe_workspace_layout", "kmoe_route", "kmoe_quantize_mx",
              "kmoe_prepare_weights", "kmoe_forward", "kmoe_forward_ex", "kmoe_device_error",
              "kmoe_selftest_wait_timeout", "kmoe_router", "kmoe_forward_router", "kmoe_selftest_activation"):
        getattr(lib, n).restype = ctypes.c_int
    return lib


_lib = load_library()


def lib():
    return _lib


def _check(fn, st):
    if st != KMOE_OK:
        raise KmoeError(fn, st, _lib)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _arg(t, name, dtype=None, shape=None, min_bytes=None):
    """Checks a caller tensor before its pointer reaches the library, which
    sees no sizes: dtype, exact shape or a minimum size in bytes, and
    contiguity.  None passes (optional arguments).  Each entry point checks
    every argument this way, then that all of them live on the GPU (_gpu)."""
    if t is None:
        return
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if min_bytes is not None and _nbytes(t) < min_bytes:
        raise ValueError(f"{name} holds {_nbytes(t)} bytes, needs at least {min_bytes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (strided input is rejected, not copied)")


def _current_gpu(stream):
    """The current GPU's number.  Launches go to it, whatever the tensors, so
    they and a given stream have to be its."""
    dev = torch.cuda.current_device()
    if stream is not None and stream.device_index != dev:
        raise ValueError(f"stream is on cuda:{stream.device_index}, the current device is cuda:{dev}")
    return dev


def _gpu(on_stream=None, **tensors):
    """Every tensor lives on the current GPU.  A given stream that uses them
    keeps them from reuse until it is through."""
    for name, t in tensors.items():
        if t is not None and not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
    dev = _current_gpu(on_stream)
    for name, t in tensors.items():
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
    if on_stream is not None:
        for t in tensors.values():
            if t is not None:
                t.record_stream(on_stream)


def _nbytes(t):
    return t.numel() * t.element_size()


def _new(shape, dtype, dev, stream):
    """An output or workspace of a call, from the memory of the stream that the
    call runs on: a block of the current stream may still be in use there when
    another stream writes it.  The current stream, where the caller goes on with
    the outputs, holds the memory from reuse too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    t.record_stream(torch.cuda.current_stream())
    return t


def _rows(t, name, ncols_name):
    """(rows, cols) of a 2-D argument."""
    if t is None or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor [rows, {ncols_name}]")
    return t.shape


KMOE_FLAG_SWIGLU = 1


def make_params(T, H, I, E, k, situ_beta=4.0, situ_linear_beta=25.0, routed_scaling_factor=1.0,
                activation="situ", swiglu_alpha=1.702, swiglu_beta=1.0, swiglu_limit=7.0):
    """`activation` is "situ" (the layer's) or "swiglu" (the clamped SwiGLU control)."""
    if activation not in ("situ", "swiglu"):
        raise ValueError(f"activation must be 'situ' or 'swiglu', got {activation!r}")
    flags = KMOE_FLAG_SWIGLU if activation == "swiglu" else 0
    return kmoe_params(T, H, I, E, k, situ_beta, situ_linear_beta, routed_scaling_factor, flags,
                       swiglu_alpha, swiglu_beta, swiglu_limit)


def kmoe_status_string(status: int) -> str:
    return _lib.kmoe_status_string(status).decode()


def kmoe_check_device(device: int = 0) -> int:
    return _lib.kmoe_check_device(device)


def kmoe_workspace_size(p: kmoe_params) -> int:
    return _lib.kmoe_workspace_size(ctypes.byref(p))


def kmoe_workspace_layout(p: kmoe_params) -> kmoe_ws_layout:
    out = kmoe_ws_layout()
    _check("kmoe_workspace_layout", _lib.kmoe_workspace_layout(ctypes.byref(p), ctypes.byref(out)))
    return out


def kmoe_route(logits, bias, k, topk_ids=None, topk_w=None, stream=None):
    T, E = _rows(logits, "logits", "E")
    _arg(logits, "logits", torch.float32)
    _arg(bias, "bias", torch.float32, (E,))
    _arg(topk_ids, "topk_ids", torch.int32, (T, k))
    _arg(topk_w, "topk_w", torch.float32, (T, k))
    _gpu(stream, logits=logits, bias=bias, topk_ids=topk_ids, topk_w=topk_w)
    if topk_ids is None:
        topk_ids = _new((T, k), torch.int32, logits.device, stream)
    if topk_w is None:
        topk_w = _new((T, k), torch.float32, logits.device, stream)
    _check("kmoe_route", _lib.kmoe_route(_ptr(logits), _ptr(bias), T, E, k, _ptr(topk_ids), _ptr(topk_w),
                                         _stream(stream)))
    return topk_ids, topk_w


def kmoe_quantize_mx(x, fmt=KMOE_MXFP8_E4M3, codes=None, scales=None, stream=None):
    rows, cols = _rows(x, "x", "cols")
    _arg(x, "x", torch.bfloat16)
    _arg(codes, "codes", torch.uint8, (rows, cols if fmt == KMOE_MXFP8_E4M3 else cols // 2))
    _arg(scales, "scales", torch.uint8, (rows, cols // 32))
    _gpu(stream, x=x, codes=codes, scales=scales)
    if codes is None:
        codes = _new((rows, cols if fmt == KMOE_MXFP8_E4M3 else cols // 2), torch.uint8, x.device, stream)
    if scales is None:
        scales = _new((rows, cols // 32), torch.uint8, x.device, stream)
    _check("kmoe_quantize_mx", _lib.kmoe_quantize_mx(_ptr(x), rows, cols, fmt, _ptr(codes), _ptr(scales),
                                                     _stream(stream)))
    return codes, scales


def kmoe_prepared_weight_bytes(p, which):
    return _lib.kmoe_prepared_weight_bytes(ctypes.byref(p), which)


def kmoe_prepare_weights(p, w13, w13_sf, w2, w2_sf, stream=None):
    """Raw checkpoint tensors -> (w13_k, w2_k) prepared weight blocks."""
    for n, t in (("w13", w13), ("w13_sf", w13_sf), ("w2", w2), ("w2_sf", w2_sf)):
        _arg(t, n, torch.uint8)
    _gpu(stream, w13=w13, w13_sf=w13_sf, w2=w2, w2_sf=w2_sf)
    if (w13.numel() != p.E * 2 * p.I * p.H // 2 or w13_sf.numel() != p.E * 2 * p.I * p.H // 32 or
            w2.numel() != p.E * p.H * p.I // 2 or w2_sf.numel() != p.E * p.H * p.I // 32):
        raise ValueError("weight sizes do not match the parameters (w13 [E, 2I, H/2], w2 [E, H, I/2])")
    a = _new(kmoe_prepared_weight_bytes(p, 0), torch.uint8, w13.device, stream)
    b = _new(kmoe_prepared_weight_bytes(p, 1), torch.uint8, w13.device, stream)
    _check("kmoe_prepare_weights", _lib.kmoe_prepare_weights(ctypes.byref(p), _ptr(w13), _ptr(w13_sf), _ptr(w2),
                                                             _ptr(w2_sf), _ptr(a), _ptr(b), _stream(stream)))
    return a, b


def _layer_args(p, x, w13_k, w2_k, out, workspace=None):
    """Checks of the arguments every forward entry point shares."""
    _arg(x, "x", torch.bfloat16, (p.T, p.H))
    _arg(w13_k, "w13_k", torch.uint8, min_bytes=kmoe_prepared_weight_bytes(p, 0))
    _arg(w2_k, "w2_k", torch.uint8, min_bytes=kmoe_prepared_weight_bytes(p, 1))
    _arg(out, "out", torch.bfloat16, (p.T, p.H))
    _arg(workspace, "workspace", torch.uint8, min_bytes=kmoe_workspace_size(p))


def kmoe_forward(p, x, logits, bias, w13_k, w2_k, topk_ids=None, topk_w=None, out=None, workspace=None,
                 stream=None, stage_events=None):
    """stage_events: optional list of 7 torch.cuda.Event recorded between the stages (kmoe_forward_ex)."""
    _layer_args(p, x, w13_k, w2_k, out, workspace)
    if topk_ids is None:
        _arg(logits, "logits", torch.float32, (p.T, p.E))
        _arg(bias, "bias", torch.float32, (p.E,))
    else:
        _arg(topk_ids, "topk_ids", torch.int32, (p.T, p.k))
        _arg(topk_w, "topk_w", torch.float32, (p.T, p.k))
    _gpu(stream, x=x, logits=logits, bias=bias, w13_k=w13_k, w2_k=w2_k, topk_ids=topk_ids, topk_w=topk_w, out=out,
         workspace=workspace)
    if out is None:
        out = _new((p.T, p.H), torch.bfloat16, x.device, stream)
    if workspace is None:
        workspace = _new(kmoe_workspace_size(p), torch.uint8, x.device, stream)
    args = (ctypes.byref(p), _ptr(x), _ptr(logits), _ptr(bias), _ptr(w13_k), _ptr(w2_k), _ptr(topk_ids),
            _ptr(topk_w), _ptr(out), _ptr(workspace), _nbytes(workspace), _stream(stream))
    if stage_events is None:
        _check("kmoe_forward", _lib.kmoe_forward(*args))
    else:
        ev = kmoe_stage_events(*[e.cuda_event for e in stage_events])
        _check("kmoe_forward_ex", _lib.kmoe_forward_ex(*args, ctypes.byref(ev)))
    return out, workspace


def kmoe_router_workspace_size(T: int, H: int, E: int) -> int:
    return _lib.kmoe_router_workspace_size(T, H, E)


def kmoe_router(x, w_gate, bias, k, logits=None, topk_ids=None, topk_w=None, workspace=None, stream=None):
    """The fused router: logits = x @ w_gate^T (bf16 operands, fp32) and the
    top-k routing of kmoe_route, in one kernel.  Returns (topk_ids, topk_w,
    logits, workspace); the workspace's first word is the device error word."""
    T, H = _rows(x, "x", "H")
    E, _ = _rows(w_gate, "w_gate", "H")
    _arg(x, "x", torch.bfloat16)
    _arg(w_gate, "w_gate", torch.bfloat16, (E, H))
    _arg(bias, "bias", torch.float32, (E,))
    _arg(logits, "logits", torch.float32, (T, E))
    _arg(topk_ids, "topk_ids", torch.int32, (T, k))
    _arg(topk_w, "topk_w", torch.float32, (T, k))
    _arg(workspace, "workspace", torch.uint8, min_bytes=kmoe_router_workspace_size(T, H, E))
    _gpu(stream, x=x, w_gate=w_gate, bias=bias, logits=logits, topk_ids=topk_ids, topk_w=topk_w, workspace=workspace)
    dev = x.device
    if logits is None:
        logits = _new((T, E), torch.float32, dev, stream)
    if topk_ids is None:
        topk_ids = _new((T, k), torch.int32, dev, stream)
    if topk_w is None:
        topk_w = _new((T, k), torch.float32, dev, stream)
    if workspace is None:
        workspace = _new(kmoe_router_workspace_size(T, H, E), torch.uint8, dev, stream)
    _check("kmoe_router", _lib.kmoe_router(_ptr(x), _ptr(w_gate), _ptr(bias), T, H, E, k, _ptr(logits),
                                           _ptr(topk_ids), _ptr(topk_w), _ptr(workspace), _nbytes(workspace),
                                           _stream(stream)))
    return topk_ids, topk_w, logits, workspace


def kmoe_forward_router(p, x, w_gate, bias, w13_k, w2_k, out=None, workspace=None, stream=None,
                        stage_events=None):
    """kmoe_forward with the fused router (routing from x and the gate weight
    instead of given logits).  stage_events: optional list of 7 torch.cuda.Event."""
    _layer_args(p, x, w13_k, w2_k, out, workspace)
    _arg(w_gate, "w_gate", torch.bfloat16, (p.E, p.H))
    _arg(bias, "bias", torch.float32, (p.E,))
    _gpu(stream, x=x, w_gate=w_gate, bias=bias, w13_k=w13_k, w2_k=w2_k, out=out, workspace=workspace)
    if out is None:
        out = _new((p.T, p.H), torch.bfloat16, x.device, stream)
    if workspace is None:
        workspace = _new(kmoe_workspace_size(p), torch.uint8, x.device, stream)
    ev = None if stage_events is None else kmoe_stage_events(*[e.cuda_event for e in stage_events])
    _check("kmoe_forward_router", _lib.kmoe_forward_router(
        ctypes.byref(p), _ptr(x), _ptr(w_gate), _ptr(bias), _ptr(w13_k), _ptr(w2_k), _ptr(out), _ptr(workspace),
        _nbytes(workspace), _stream(stream), None if ev is None else ctypes.byref(ev)))
    return out, workspace


def kmoe_forward_noalloc(p, x, logits, bias, w13_k, w2_k, topk_ids=None, topk_w=None, out=None,
                         device_error=None, stream=None):
    """kmoe_forward without a workspace argument, for hosts that cannot
    allocate device memory: the library's built-in scratch array
    (NOALLOC_SCRATCH_BYTES, shared by all calls) is used instead.  `out` and
    the optional `device_error` (one int32 on the device) are caller-owned."""
    _layer_args(p, x, w13_k, w2_k, out)
    if topk_ids is None:
        _arg(logits, "logits", torch.float32, (p.T, p.E))
        _arg(bias, "bias", torch.float32, (p.E,))
    else:
        _arg(topk_ids, "topk_ids", torch.int32, (p.T, p.k))
        _arg(topk_w, "topk_w", torch.float32, (p.T, p.k))
    _arg(device_error, "device_error", min_bytes=4)
    _gpu(stream, x=x, logits=logits, bias=bias, w13_k=w13_k, w2_k=w2_k, topk_ids=topk_ids, topk_w=topk_w, out=out,
         device_error=device_error)
    if out is None:
        out = _new((p.T, p.H), torch.bfloat16, x.device, stream)
    _check("kmoe_forward_noalloc", _lib.kmoe_forward_noalloc(
        ctypes.byref(p), _ptr(x), _ptr(logits), _ptr(bias), _ptr(w13_k), _ptr(w2_k), _ptr(topk_ids), _ptr(topk_w),
        _ptr(out), _ptr(device_error), _stream(stream)))
    return out


def kmoe_forward_mx(p, x_codes, x_scales, topk_ids, topk_w, w13_k, w2_k, out=None, workspace=None, stream=None):
    """kmoe_forward on rows quantised before (kmoe_rmsnorm's or
    kmoe_quantize_mx's codes [T, H] and scales [T, H/32]), routing given."""
    dev = _rows_on(x_codes, "x_codes", "H")[2]
    _args(stream, dev, (("x_codes", x_codes, torch.uint8, (p.T, p.H)),
                        ("x_scales", x_scales, torch.uint8, (p.T, p.H // 32)),
                        ("topk_ids", topk_ids, torch.int32, (p.T, p.k)),
                        ("topk_w", topk_w, torch.float32, (p.T, p.k)), ("out", out, torch.bfloat16, (p.T, p.H))))
    _arg(w13_k, "w13_k", torch.uint8, min_bytes=kmoe_prepared_weight_bytes(p, 0))
    _arg(w2_k, "w2_k", torch.uint8, min_bytes=kmoe_prepared_weight_bytes(p, 1))
    _arg(workspace, "workspace", torch.uint8, min_bytes=kmoe_workspace_size(p))
    _gpu(stream, w13_k=w13_k, w2_k=w2_k, workspace=workspace)
    if out is None:
        out = _new((p.T, p.H), torch.bfloat16, dev, stream)
    if workspace is None:
        workspace = _new(kmoe_workspace_size(p), torch.uint8, dev, stream)
    _check("kmoe_forward_mx", _lib.kmoe_forward_mx(
        ctypes.byref(p), _ptr(x_codes), _ptr(x_scales), _ptr(topk_ids), _ptr(topk_w), _ptr(w13_k), _ptr(w2_k),
        _ptr(out), _ptr(workspace), _nbytes(workspace), _raw_stream(dev, stream)))
    return out, workspace


# ---- the operators around the experts.  Decode calls are a few microseconds
# on the GPU, so their argument checks are one pass over the tensors.

def _args(stream, dev, named):
    """Checks (name, tensor, dtype, shape) of each argument, None passing, on
    the current GPU, whose number `dev` has to be, and returns their addresses.
    The errors are _arg's and _gpu's.  A tensor that a given stream uses is kept
    from reuse until that stream is through."""
    at = []
    for name, t, dtype, shape in named:
        if t is None:
            at.append(None)
        elif t.dtype is dtype and t.shape == shape and t.get_device() == dev >= 0 and t.is_contiguous():
            at.append(t.data_ptr())
        else:
            for n, u, d, s in named:
                _arg(u, n, d, s)
            _gpu(stream, **{n: u for n, u, _, _ in named})
            at.append(t.data_ptr())
    if stream is not None or dev != _current_device():
        _gpu(stream, **{n: u for n, u, _, _ in named})
    return at


# None in a torch without CUDA, where no call gets past its checks
_current_device = getattr(torch._C, "_cuda_getDevice", None)  # torch.cuda.current_device without its 0.3 us
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# scratch of one call, from the caching allocator without a tensor around it (a
# tensor costs about 5 us beside a launch)
_scratch_alloc = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", None)
_scratch_free = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", None)


def _raw_stream(dev, stream):
    return _current_stream(dev) if stream is None else stream.cuda_stream


def _rows_on(t, name, ncols_name):
    """(rows, cols, device ordinal) of a 2-D argument."""
    if t is None or t.dim() != 2:
        _rows(t, name, ncols_name)
    rows, cols = t.shape
    return rows, cols, t.get_device()


KMOE_NORM_STREAM_F32 = 1
KMOE_NORM_WEIGHT_F32 = 2
_F32_OR_BF16 = (torch.bfloat16, torch.float32)


def _type_of(t, name, default):
    if t is None:
        return default
    if t.dtype not in _F32_OR_BF16:
        raise ValueError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    return t.dtype


def kmoe_rmsnorm(x, weight, residual=None, eps=1e-6, mx=False, h=None, y=None, codes=None, scales=None, stream=None):
    """h = x + residual, y = rmsnorm(h) * weight and, with `mx`, the MXFP8 codes
    and scales of y, in one kernel.  Returns (h, y, codes, scales); h is None
    without a residual, codes and scales without `mx`.  residual and h are
    bf16 or fp32 (h may be residual itself), weight bf16 or fp32."""
    T, H, dev = _rows_on(x, "x", "H")
    st = _type_of(residual, "residual", torch.bfloat16)
    wt = _type_of(weight, "weight", None)
    if h is not None and residual is None:
        raise ValueError("h needs a residual")
    if not mx and (codes is not None or scales is not None):
        raise ValueError("codes and scales need mx=True")
    rows = (T, H)
    at = _args(stream, dev, (("x", x, torch.bfloat16, rows), ("residual", residual, st, rows),
                             ("weight", weight, wt, (H,)), ("h", h, st, rows), ("y", y, torch.bfloat16, rows),
                             ("codes", codes, torch.uint8, rows), ("scales", scales, torch.uint8, (T, H // 32))))
    if h is None and residual is not None:
        h = _new(rows, st, dev, stream)
        at[3] = h.data_ptr()
    if y is None:
        y = _new(rows, torch.bfloat16, dev, stream)
        at[4] = y.data_ptr()
    if mx:
        if codes is None:
            codes = _new(rows, torch.uint8, dev, stream)
            at[5] = codes.data_ptr()
        if scales is None:
            scales = _new((T, H // 32), torch.uint8, dev, stream)
            at[6] = scales.data_ptr()
    flags = (KMOE_NORM_STREAM_F32 if st is torch.float32 else 0) | (KMOE_NORM_WEIGHT_F32 if wt is torch.float32 else 0)
    _check("kmoe_rmsnorm", _lib.kmoe_rmsnorm(at[0], at[1], at[2], T, H, eps, flags, at[3], at[4], at[5], at[6],
                                             _raw_stream(dev, stream)))
    return h, y, codes, scales


def kmoe_rmsnorm_workspace_size(T: int, H: int) -> int:
    return _lib.kmoe_rmsnorm_workspace_size(T, H)


def kmoe_rmsnorm_backward(dy, h, weight, dh_in=None, eps=1e-6, dh=None, dweight=None, workspace=None, stream=None):
    """Gradient of kmoe_rmsnorm at the stored h: (dh, dweight), dh of h's type
    (the gradient of x and of residual alike, with dh_in added), dweight fp32.
    dh may be dh_in itself."""
    T, H, dev = _rows_on(h, "h", "H")
    st = _type_of(h, "h", None)
    wt = _type_of(weight, "weight", None)
    rows = (T, H)
    at = _args(stream, dev, (("dy", dy, torch.bfloat16, rows), ("h", h, st, rows), ("weight", weight, wt, (H,)),
                             ("dh_in", dh_in, st, rows), ("dh", dh, st, rows),
                             ("dweight", dweight, torch.float32, (H,))))
    n = _lib.kmoe_rmsnorm_workspace_size(T, H)
    if workspace is not None:
        _arg(workspace, "workspace", torch.uint8, min_bytes=n)
        _gpu(stream, workspace=workspace)
    if dh is None:
        dh = _new(rows, st, dev, stream)
        at[4] = dh.data_ptr()
    if dweight is None:
        dweight = _new((H,), torch.float32, dev, stream)
        at[5] = dweight.data_ptr()
    flags = (KMOE_NORM_STREAM_F32 if st is torch.float32 else 0) | (KMOE_NORM_WEIGHT_F32 if wt is torch.float32 else 0)
    raw = _raw_stream(dev, stream)
    # freed when the launches are queued: the memory's next user on this stream comes after them
    scratch = _scratch_alloc(max(n, 1), raw) if workspace is None else 0
    try:
        _check("kmoe_rmsnorm_backward", _lib.kmoe_rmsnorm_backward(
            at[0], at[1], at[2], at[3], T, H, eps, flags, at[4], at[5], scratch or workspace.data_ptr(), n, raw))
    finally:
        if scratch:
            _scratch_free(scratch)
    return dh, dweight


KMOE_ROUTE_SOFTMAX = 1
KMOE_ROUTE_RENORMALIZE = 2
_SCORES = {"sigmoid": 0, "softmax": KMOE_ROUTE_SOFTMAX}


@functools.lru_cache(maxsize=256)
def _route_params(T, E, k, n_group, topk_group, score, renormalize, scale):
    """The C struct of these parameters (read only, so calls can share it)."""
    if score not in _SCORES:
        raise ValueError(f"score must be 'sigmoid' or 'softmax', got {score!r}")
    return ctypes.byref(kmoe_route_params(T, E, k, n_group, topk_group,
                                          _SCORES[score] | (KMOE_ROUTE_RENORMALIZE if renormalize else 0), scale))


def kmoe_route_grouped(logits, bias, k, score="sigmoid", n_group=1, topk_group=1, renormalize=True, scale=1.0,
                       topk_ids=None, topk_w=None, stream=None):
    """Top-k routing with sigmoid or softmax scores, an optional balance bias
    (None: the logits choose), `topk_group` of `n_group` expert groups and
    optionally renormalised weights.  Returns (topk_ids, topk_w); slots no
    expert could fill hold id -1 and weight 0."""
    T, E, dev = _rows_on(logits, "logits", "E")
    at = _args(stream, dev, (("logits", logits, torch.float32, (T, E)), ("bias", bias, torch.float32, (E,)),
                             ("topk_ids", topk_ids, torch.int32, (T, k)), ("topk_w", topk_w, torch.float32, (T, k))))
    p = _route_params(T, E, k, n_group, topk_group, score, renormalize, scale)
    if topk_ids is None:
        topk_ids = _new((T, k), torch.int32, dev, stream)
        at[2] = topk_ids.data_ptr()
    if topk_w is None:
        topk_w = _new((T, k), torch.float32, dev, stream)
        at[3] = topk_w.data_ptr()
    _check("kmoe_route_grouped", _lib.kmoe_route_grouped(p, at[0], at[1], at[2], at[3], _raw_stream(dev, stream)))
    return topk_ids, topk_w


def kmoe_route_backward(d_w, logits, topk_ids, score="sigmoid", renormalize=True, scale=1.0, d_logits=None,
                        stream=None):
    """Gradient of the routing weights with respect to the logits: d_logits
    fp32 [T, E], dense, for the ids that were chosen."""
    T, E, dev = _rows_on(logits, "logits", "E")
    k = _rows(topk_ids, "topk_ids", "k")[1]
    at = _args(stream, dev, (("d_w", d_w, torch.float32, (T, k)), ("logits", logits, torch.float32, (T, E)),
                             ("topk_ids", topk_ids, torch.int32, (T, k)),
                             ("d_logits", d_logits, torch.float32, (T, E))))
    p = _route_params(T, E, k, 1, 1, score, renormalize, scale)
    if d_logits is None:
        d_logits = _new((T, E), torch.float32, dev, stream)
        at[3] = d_logits.data_ptr()
    _check("kmoe_route_backward", _lib.kmoe_route_backward(p, at[0], at[1], at[2], at[3], _raw_stream(dev, stream)))
    return d_logits


def kmoe_combine_backward(d_out, y, topk_ids, E, routed_scaling_factor=1.0, d_w=None, stream=None):
    """Gradient of the combine with respect to the routing weights: fp32
    [T, k] from d_out bf16 [T, H] and the per-slot outputs y fp32 [T*k, H]
    that a forward leaves in its workspace (stage_views(p, ws)["y"])."""
    T, H, dev = _rows_on(d_out, "d_out", "H")
    k = _rows(topk_ids, "topk_ids", "k")[1]
    at = _args(stream, dev, (("d_out", d_out, torch.bfloat16, (T, H)), ("y", y, torch.float32, (T * k, H)),
                             ("topk_ids", topk_ids, torch.int32, (T, k)), ("d_w", d_w, torch.float32, (T, k))))
    if d_w is None:
        d_w = _new((T, k), torch.float32, dev, stream)
        at[3] = d_w.data_ptr()
    _check("kmoe_combine_backward", _lib.kmoe_combine_backward(at[0], at[1], at[2], T, H, k, E, routed_scaling_factor,
                                                               at[3], _raw_stream(dev, stream)))
    return d_w


def kmoe_selftest_activation(p, gate, up, out=None, stream=None):
    """The FC1 epilogue's activation of (gate, up), elementwise (fp32 device
    arrays of one shape), by the forward's own device functions."""
    _arg(gate, "gate", torch.float32, tuple(gate.shape))
    _arg(up, "up", torch.float32, tuple(gate.shape))
    _arg(out, "out", torch.float32, tuple(gate.shape))
    _gpu(stream, gate=gate, up=up, out=out)
    if out is None:
        out = _new(tuple(gate.shape), torch.float32, gate.device, stream)
    _check("kmoe_selftest_activation", _lib.kmoe_selftest_activation(
        ctypes.byref(p), _ptr(gate), _ptr(up), gate.numel(), _ptr(out), _stream(stream)))
    return out


def kmoe_device_error(workspace, stream=None):
    _arg(workspace, "workspace", min_bytes=4)
    _gpu(stream, workspace=workspace)
    word = ctypes.c_uint32(0)
    st = _lib.kmoe_device_error(_ptr(workspace), ctypes.byref(word), _stream(stream))
    return st, word.value


def kmoe_tile_sf_offset(tile, local_row, g, tile_rows, K, max_tiles):
    return _lib.kmoe_tile_sf_offset(tile, local_row, g, tile_rows, K, max_tiles)


def kmoe_mma_peak_run(iters, N, workspace, stream=None):
    """Launch the tensor-pipe roof kernel; returns the launch's FLOP count."""
    _arg(workspace, "workspace", min_bytes=4)
    _gpu(stream, workspace=workspace)
    _check("kmoe_mma_peak_run", _lib.kmoe_mma_peak_run(iters, N, _ptr(workspace), _stream(stream)))
    sms = torch.cuda.get_device_properties(workspace.device).multi_processor_count
    return sms * iters * 4 * 2 * 128 * N * 32


def kmoe_selftest_wait_timeout(workspace, budget_us, stream=None):
    _arg(workspace, "workspace", min_bytes=4)
    _gpu(stream, workspace=workspace)
    _check("kmoe_selftest_wait_timeout",
           _lib.kmoe_selftest_wait_timeout(_ptr(workspace), budget_us, _stream(stream)))


def stage_views(p, workspace):
    """Views of the stage tensors kmoe_forward leaves in the workspace."""
    L = kmoe_workspace_layout(p)
    R = p.T * p.k

    def v(off, n, dtype):
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        return workspace[off:off + nbytes].view(dtype)

    return {
        "layout": L,
        "topk_ids": v(L.topk_ids, R, torch.int32).view(p.T, p.k),
        "topk_w": v(L.topk_w, R, torch.float32).view(p.T, p.k),
        "counts": v(L.counts, p.E, torch.int32),
        "seg_start": v(L.seg_start, p.E + 1, torch.int32),
        "tile_start": v(L.tile_start, p.E + 1, torch.int32),
        "row_of_slot": v(L.row_of_slot, R, torch.int32),
        "slot_of_row": v(L.slot_of_row, R, torch.int32),
        "xq": v(L.xq, R * p.H, torch.uint8).view(R, p.H),
        "iq": v(L.iq, R * p.I, torch.uint8).view(R, p.I),
        "xsf": workspace[L.xsf:L.xsf + (p.H // 128) * L.max_tiles * ((L.tile_rows + 127) // 128) * 512],
        "isf": workspace[L.isf:L.isf + (p.I // 128) * L.max_tiles * ((L.tile_rows + 127) // 128) * 512],
        "tile_start_big": v(L.tile_start_big, p.E + 1, torch.int32),
        "xsf_big": workspace[L.xsf_big:L.xsf_big + (p.H // 128) * L.max_tiles_big * 2 * 512],
        "isf_big": workspace[L.isf_big:L.isf_big + (p.I // 128) * L.max_tiles_big * 2 * 512],
        "y": v(L.y, R * p.H, torch.float32).view(R, p.H),
        "logits": v(L.logits, p.T * p.E, torch.float32).view(p.T, p.E),
    }


from .products import *  # noqa: E402,F401,F403  (the expert products in 8 bits; they use what is above)
