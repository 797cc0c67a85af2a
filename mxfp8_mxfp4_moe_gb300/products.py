"""Expert products in 8 bits (include/kmoe_products.h): the tokens' rows sorted by
expert and summed back with their weights, quantisation to E4M3 with a scale for
each block of 128, products of such operands, and the gradients of each.

Part of the package's binding, whose rules for arguments, streams and memory
hold here; the functions are the package's own (kmoe_gemm_fp8 and so on).  Codes
are torch.uint8: a checkpoint's torch.float8_e4m3fn tensor goes in as its
.view(torch.uint8), and codes are values as .view(torch.float8_e4m3fn).
"""
from __future__ import annotations

import ctypes

import torch

import mxfp8_mxfp4_moe_gb300 as _k
from mxfp8_mxfp4_moe_gb300 import (_F32_OR_BF16, _arg, _args, _check, _gpu, _new, _raw_stream, _rows,
                                   _rows_on, _type_of)

PRODUCT_EXPORTS = ("kmoe_sort_workspace_size", "kmoe_sort_tokens", "kmoe_permute", "kmoe_unpermute",
                   "kmoe_unpermute_backward", "kmoe_quantize_fp8_workspace_size", "kmoe_quantize_fp8",
                   "kmoe_quantize_fp8_weights", "kmoe_fp8_padded_rows", "kmoe_quantize_fp8_cols", "kmoe_gemm_fp8",
                   "kmoe_gemm_fp8_wgrad")

__all__ = ["PRODUCT_EXPORTS", "KMOE_ROWS_F32", "KMOE_OUT_F32", "KMOE_GEMM_TRANSPOSE", "KMOE_GEMM_OUT_F32",
           "GEMM_FP8_WORKSPACE_BYTES", *PRODUCT_EXPORTS]

KMOE_ROWS_F32 = 1
KMOE_OUT_F32 = 2
KMOE_GEMM_TRANSPOSE = 1
KMOE_GEMM_OUT_F32 = 2
GEMM_FP8_WORKSPACE_BYTES = 256
_BLOCK = 128  # values a scale
_U8, _I32, _F32, _BF16 = torch.uint8, torch.int32, torch.float32, torch.bfloat16


def _declare(lib):
    P, S, I, V, U = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_void_p, ctypes.c_uint32
    for name, args in (("kmoe_sort_workspace_size", [I, I, I]),
                       ("kmoe_sort_tokens", [P, I, I, I, P, P, P, P, S, V]),
                       ("kmoe_permute", [P, P, I, I, I, U, P, V]),
                       ("kmoe_unpermute", [P, P, P, I, I, I, U, P, V]),
                       ("kmoe_unpermute_backward", [P, P, P, P, I, I, I, U, P, P, V]),
                       ("kmoe_quantize_fp8_workspace_size", [I, I, I]),
                       ("kmoe_quantize_fp8", [P, I, I, P, I, P, P, P, S, V]),
                       ("kmoe_quantize_fp8_weights", [P, I, I, I, P, P, V]),
                       ("kmoe_fp8_padded_rows", [I, I]),
                       ("kmoe_quantize_fp8_cols", [P, I, I, P, I, P, P, V]),
                       ("kmoe_gemm_fp8", [P, P, P, P, P, I, I, I, I, U, P, P, S, V]),
                       ("kmoe_gemm_fp8_wgrad", [P, P, P, P, P, I, I, I, I, P, P, S, V])):
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = S if name.endswith("_size") else I


_declare(_k._lib)


def kmoe_sort_workspace_size(T: int, E: int, k: int) -> int:
    return _k._lib.kmoe_sort_workspace_size(T, E, k)


def kmoe_sort_tokens(topk_ids, E, row_of_slot=None, slot_of_row=None, seg_start=None, workspace=None, stream=None):
    """The slots of topk_ids [T, k] int32 sorted by expert (stable).  Returns
    (row_of_slot [T, k], slot_of_row [T * k], seg_start [E + 1]), int32: a slot's
    sorted row (-1 for ids outside [0, E)), a row's slot (-1 past the last row)
    and each expert's first row."""
    T, k, dev = _rows_on(topk_ids, "topk_ids", "k")
    at = _args(stream, dev, (("topk_ids", topk_ids, _I32, (T, k)), ("row_of_slot", row_of_slot, _I32, (T, k)),
                             ("slot_of_row", slot_of_row, _I32, (T * k,)), ("seg_start", seg_start, _I32, (E + 1,))))
    n = _k._lib.kmoe_sort_workspace_size(T, E, k)
    if workspace is not None:
        _arg(workspace, "workspace", _U8, min_bytes=n)
        _gpu(stream, workspace=workspace)
    if row_of_slot is None:
        row_of_slot = _new((T, k), _I32, dev, stream)
        at[1] = row_of_slot.data_ptr()
    if slot_of_row is None:
        slot_of_row = _new((T * k,), _I32, dev, stream)
        at[2] = slot_of_row.data_ptr()
    if seg_start is None:
        seg_start = _new((max(E, 0) + 1,), _I32, dev, stream)
        at[3] = seg_start.data_ptr()
    raw = _raw_stream(dev, stream)
    # freed when the launches are queued: the memory's next user on this stream comes after them
    scratch = _k._scratch_alloc(max(n, 1), raw) if workspace is None else 0
    try:
        _check("kmoe_sort_tokens", _k._lib.kmoe_sort_tokens(at[0], T, E, k, at[1], at[2], at[3],
                                                            scratch or workspace.data_ptr(), n, raw))
    finally:
        if scratch:
            _k._scratch_free(scratch)
    return row_of_slot, slot_of_row, seg_start


def _row_flags(rows, tokens):
    return (KMOE_ROWS_F32 if rows is _F32 else 0) | (KMOE_OUT_F32 if tokens is _F32 else 0)


def kmoe_permute(x, row_of_slot, out=None, stream=None):
    """out[row_of_slot[t, j]] = x[t]: the tokens' rows [T, H] (bf16 or fp32) in
    sorted order [T * k, H].  Rows without a slot are left as they were.  Its
    gradient is kmoe_unpermute without weights."""
    T, H, dev = _rows_on(x, "x", "H")
    k = _rows(row_of_slot, "row_of_slot", "k")[1]
    ty = _type_of(x, "x", None)
    at = _args(stream, dev, (("x", x, ty, (T, H)), ("row_of_slot", row_of_slot, _I32, (T, k)),
                             ("out", out, ty, (T * k, H))))
    if out is None:
        out = _new((T * k, H), ty, dev, stream)
        at[2] = out.data_ptr()
    _check("kmoe_permute", _k._lib.kmoe_permute(at[0], at[1], T, H, k, _row_flags(ty, _BF16), at[2],
                                                _raw_stream(dev, stream)))
    return out


def _out_type(out, out_dtype):
    ty = out_dtype if out is None else _type_of(out, "out", None)
    if ty not in _F32_OR_BF16:
        raise ValueError(f"out_dtype must be torch.bfloat16 or torch.float32, got {ty}")
    return ty


def kmoe_unpermute(y, row_of_slot, topk_w=None, out=None, out_dtype=torch.bfloat16, stream=None):
    """out[t] = sum_j topk_w[t, j] * y[row_of_slot[t, j]] (without weights: the
    sum of the rows).  y [T * k, H] bf16 or fp32, out [T, H] of `out`'s type or
    out_dtype."""
    T, k = _rows(row_of_slot, "row_of_slot", "k")
    _, H, dev = _rows_on(y, "y", "H")
    ty, to = _type_of(y, "y", None), _out_type(out, out_dtype)
    at = _args(stream, dev, (("y", y, ty, (T * k, H)), ("row_of_slot", row_of_slot, _I32, (T, k)),
                             ("topk_w", topk_w, _F32, (T, k)), ("out", out, to, (T, H))))
    if out is None:
        out = _new((T, H), to, dev, stream)
        at[3] = out.data_ptr()
    _check("kmoe_unpermute", _k._lib.kmoe_unpermute(at[0], at[1], at[2], T, H, k, _row_flags(ty, to), at[3],
                                                    _raw_stream(dev, stream)))
    return out


def kmoe_unpermute_backward(d_out, y, row_of_slot, topk_w, d_y=None, d_w=None, stream=None):
    """Gradient of kmoe_unpermute: (d_y, d_w), d_y [T * k, H] of y's type (may be
    y itself; rows without a slot are left as they were), d_w fp32 [T, k].
    d_out [T, H] and y are bf16 or fp32."""
    T, H, dev = _rows_on(d_out, "d_out", "H")
    k = _rows(row_of_slot, "row_of_slot", "k")[1]
    tg, ty = _type_of(d_out, "d_out", None), _type_of(y, "y", None)
    at = _args(stream, dev, (("d_out", d_out, tg, (T, H)), ("y", y, ty, (T * k, H)),
                             ("row_of_slot", row_of_slot, _I32, (T, k)), ("topk_w", topk_w, _F32, (T, k)),
                             ("d_y", d_y, ty, (T * k, H)), ("d_w", d_w, _F32, (T, k))))
    if d_y is None:
        d_y = _new((T * k, H), ty, dev, stream)
        at[4] = d_y.data_ptr()
    if d_w is None:
        d_w = _new((T, k), _F32, dev, stream)
        at[5] = d_w.data_ptr()
    _check("kmoe_unpermute_backward", _k._lib.kmoe_unpermute_backward(
        at[0], at[1], at[2], at[3], T, H, k, _row_flags(ty, tg), at[4], at[5], _raw_stream(dev, stream)))
    return d_y, d_w


def kmoe_quantize_fp8_workspace_size(rows: int, cols: int, k: int = 1) -> int:
    return _k._lib.kmoe_quantize_fp8_workspace_size(rows, cols, k)


def kmoe_quantize_fp8(x, row_of_slot=None, codes=None, scales=None, workspace=None, stream=None):
    """E4M3 codes [rows, cols] and fp32 power-of-two scales [ceil(cols/128), rows]
    of bf16 rows, one scale for 128 columns of a row.  With row_of_slot [T, k]
    token t's row goes to the sorted rows of its slots: codes [T * k, cols]."""
    T, H, dev = _rows_on(x, "x", "cols")
    k = 1 if row_of_slot is None else _rows(row_of_slot, "row_of_slot", "k")[1]
    sf = (-(-H // _BLOCK), T * k)
    at = _args(stream, dev, (("x", x, _BF16, (T, H)), ("row_of_slot", row_of_slot, _I32, (T, k)),
                             ("codes", codes, _U8, (T * k, H)), ("scales", scales, _F32, sf)))
    n = 0 if row_of_slot is None else _k._lib.kmoe_quantize_fp8_workspace_size(T, H, k)
    if workspace is not None:
        _arg(workspace, "workspace", _U8, min_bytes=n)
        _gpu(stream, workspace=workspace)
    if codes is None:
        codes = _new((T * k, H), _U8, dev, stream)
        at[2] = codes.data_ptr()
    if scales is None:
        scales = _new(sf, _F32, dev, stream)
        at[3] = scales.data_ptr()
    raw = _raw_stream(dev, stream)
    # freed when the launches are queued: the memory's next user on this stream comes after them
    scratch = _k._scratch_alloc(n, raw) if n and workspace is None else 0
    try:
        _check("kmoe_quantize_fp8", _k._lib.kmoe_quantize_fp8(
            at[0], T, H, at[1], k, at[2], at[3], scratch or (workspace.data_ptr() if n else None), n, raw))
    finally:
        if scratch:
            _k._scratch_free(scratch)
    return codes, scales


def _weights(w, name):
    """(E, N, K) of weights [E, N, K], or [N, K] for a dense projection, and their scales' shape."""
    s = () if w is None else w.shape
    if len(s) == 3:
        E, N, K = s
        return s, (E, (N + 127) // 128, (K + 127) // 128)
    if len(s) != 2:
        raise ValueError(f"{name} must be a tensor [E, N, K] or [N, K]")
    N, K = s
    return (1, N, K), ((N + 127) // 128, (K + 127) // 128)


def kmoe_quantize_fp8_weights(w, codes=None, scales=None, stream=None):
    """E4M3 codes and fp32 power-of-two scales [.., ceil(N/128), ceil(K/128)] of
    bf16 weights [E, N, K] or [N, K], one scale for a block of 128 x 128."""
    (E, N, K), sf = _weights(w, "w")
    dev = w.get_device()
    at = _args(stream, dev, (("w", w, _BF16, w.shape), ("codes", codes, _U8, w.shape), ("scales", scales, _F32, sf)))
    if codes is None:
        codes = _new(tuple(w.shape), _U8, dev, stream)
        at[1] = codes.data_ptr()
    if scales is None:
        scales = _new(sf, _F32, dev, stream)
        at[2] = scales.data_ptr()
    _check("kmoe_quantize_fp8_weights", _k._lib.kmoe_quantize_fp8_weights(at[0], E, N, K, at[1], at[2],
                                                                          _raw_stream(dev, stream)))
    return codes, scales


def kmoe_fp8_padded_rows(rows: int, E: int) -> int:
    return _k._lib.kmoe_fp8_padded_rows(rows, E)


def _experts(seg_start):
    """Experts of a product, and its segments' entry for _args; None: one expert."""
    if seg_start is not None and (seg_start.dim() != 1 or seg_start.shape[0] < 2):
        raise ValueError("seg_start must be a 1-D tensor [E + 1]")
    E = 1 if seg_start is None else seg_start.shape[0] - 1
    return E, ("seg_start", seg_start, _I32, (E + 1,))


def kmoe_quantize_fp8_cols(x, seg_start=None, codes=None, scales=None, stream=None):
    """E4M3 codes [P, cols] and fp32 power-of-two scales [P/128, cols] of bf16
    rows for kmoe_gemm_fp8_wgrad, one scale for 128 rows of a column; every
    expert's rows start on a multiple of 128 (P = kmoe_fp8_padded_rows(rows, E))."""
    R, F, dev = _rows_on(x, "x", "cols")
    E, seg = _experts(seg_start)
    P = max(_k._lib.kmoe_fp8_padded_rows(R, E), 0)  # sizes that it refuses the call refuses too
    at = _args(stream, dev, (("x", x, _BF16, (R, F)), seg, ("codes", codes, _U8, (P, F)),
                             ("scales", scales, _F32, (P // _BLOCK, F))))
    if codes is None:
        codes = _new((P, F), _U8, dev, stream)
        at[2] = codes.data_ptr()
    if scales is None:
        scales = _new((P // _BLOCK, F), _F32, dev, stream)
        at[3] = scales.data_ptr()
    _check("kmoe_quantize_fp8_cols", _k._lib.kmoe_quantize_fp8_cols(at[0], R, F, at[1], E, at[2], at[3],
                                                                    _raw_stream(dev, stream)))
    return codes, scales


def _workspace_entry(workspace):
    """A product's workspace, for _args."""
    if workspace is None:
        return "workspace", None, _U8, None
    if workspace.numel() < GEMM_FP8_WORKSPACE_BYTES:
        _arg(workspace, "workspace", _U8, min_bytes=GEMM_FP8_WORKSPACE_BYTES)
    return "workspace", workspace, _U8, workspace.shape


def kmoe_gemm_fp8(x, x_scales, w, w_scales, seg_start=None, transpose=False, out=None, out_dtype=torch.bfloat16,
                  workspace=None, stream=None):
    """Rows x [M, K] times weights w [E, N, K] (or [N, K]) transposed, out [M, N];
    with `transpose` rows x [M, N] times w, out [M, K] (the rows' gradient).  x
    and x_scales as kmoe_quantize_fp8 gives them, w_scales [E, ceil(N/128),
    ceil(K/128)] fp32.  Expert e's rows are [seg_start[e], seg_start[e+1]); rows
    outside are left as they were.  Returns (out, workspace); the workspace's
    first word is the device error word, which the next product in it clears:
    read it before (kmoe_device_error), or let each product have its own."""
    M, _, dev = _rows_on(x, "x", "cols")
    (E, N, K), sf = _weights(w, "w")
    experts, seg = _experts(seg_start)
    if experts != E:
        raise ValueError(f"w holds {E} experts, seg_start {experts}")
    wide, F = (N, K) if transpose else (K, N)
    to = _out_type(out, out_dtype)
    at = _args(stream, dev, (("x", x, _U8, (M, wide)), ("x_scales", x_scales, _F32, (-(-wide // _BLOCK), M)),
                             ("w", w, _U8, w.shape), ("w_scales", w_scales, _F32, sf), seg, ("out", out, to, (M, F)),
                             _workspace_entry(workspace)))
    if workspace is None:
        workspace = _new(GEMM_FP8_WORKSPACE_BYTES, _U8, dev, stream)
        at[6] = workspace.data_ptr()
        if M == 0:  # a call without rows leaves the error word as it is
            with torch.cuda.stream(stream):
                workspace.zero_()
    if out is None:
        out = _new((M, F), to, dev, stream)
        at[5] = out.data_ptr()
    flags = (KMOE_GEMM_TRANSPOSE if transpose else 0) | (KMOE_GEMM_OUT_F32 if to is _F32 else 0)
    _check("kmoe_gemm_fp8", _k._lib.kmoe_gemm_fp8(at[0], at[1], at[2], at[3], at[4], M, N, K, E, flags, at[5],
                                                  at[6], workspace.numel(), _raw_stream(dev, stream)))
    return out, workspace


def kmoe_gemm_fp8_wgrad(dy, dy_scales, x, x_scales, seg_start=None, dw=None, workspace=None, stream=None):
    """The weights' gradient fp32 [E, N, K] ([1, N, K] without seg_start) of
    kmoe_gemm_fp8, from dy [P, N] and x [P, K] as kmoe_quantize_fp8_cols gives
    them for the same rows and seg_start.  Returns (dw, workspace)."""
    P, N, dev = _rows_on(dy, "dy", "N")
    K = _rows(x, "x", "K")[1]
    E, seg = _experts(seg_start)
    at = _args(stream, dev, (("dy", dy, _U8, (P, N)), ("dy_scales", dy_scales, _F32, (P // _BLOCK, N)),
                             ("x", x, _U8, (P, K)), ("x_scales", x_scales, _F32, (P // _BLOCK, K)), seg,
                             ("dw", dw, _F32, (E, N, K)), _workspace_entry(workspace)))
    if workspace is None:
        workspace = _new(GEMM_FP8_WORKSPACE_BYTES, _U8, dev, stream)
        at[6] = workspace.data_ptr()
    if dw is None:
        dw = _new((E, N, K), _F32, dev, stream)
        at[5] = dw.data_ptr()
    _check("kmoe_gemm_fp8_wgrad", _k._lib.kmoe_gemm_fp8_wgrad(
        at[0], at[1], at[2], at[3], at[4], P, N, K, E, at[5], at[6], workspace.numel(),
        _raw_stream(dev, stream)))
    return dw, workspace
