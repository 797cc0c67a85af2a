"""CPU checks of the sort by expert, the block-scaled quantisers and products: the
oracle by hand, and the refusals of the C entry points and of the binding."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import mxfp8_mxfp4_moe_gb300 as K
from oracle import formats as F
from oracle import products as P

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ARG, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 5


# ---------------------------------------------------------------- the oracle


def test_sort_by_hand():
    row, slot, seg = P.sort_tokens(np.array([[2, 0], [0, -1], [2, 2], [7, 1]]), 3)
    assert row.tolist() == [[3, 0], [1, -1], [4, 5], [-1, 2]]
    assert slot.tolist() == [1, 2, 7, 0, 4, 5, -1, -1] and seg.tolist() == [0, 2, 3, 6]


def test_unpermute_and_its_gradient_by_hand():
    y = np.array([[1.0, 2.0], [3.0, 5.0], [7.0, 11.0]])
    rows, w = np.array([[2, -1], [0, 1]]), np.array([[0.5, 9.0], [2.0, -1.0]])
    assert P.unpermute(y, rows, w)[0].tolist() == [[3.5, 5.5], [-1.0, -1.0]]
    assert P.unpermute(y, rows)[0].tolist() == [[7.0, 11.0], [4.0, 7.0]]
    d_y, d_w, _ = P.unpermute_backward(np.array([[1.0, 10.0], [100.0, 1000.0]]), y, rows, w)
    assert d_y.tolist() == [[200.0, 2000.0], [-100.0, -1000.0], [0.5, 5.0]]
    assert d_w.tolist() == [[117.0, 0.0], [2100.0, 5300.0]]


def test_unpermute_gradient_against_differences():
    g = np.random.default_rng(0)
    y, w, d_out = g.standard_normal((12, 5)), g.standard_normal((4, 3)), g.standard_normal((4, 5))
    rows = g.permutation(12).reshape(4, 3)
    rows[1, 2] = -1
    d_y, d_w, _ = P.unpermute_backward(d_out, y, rows, w)
    for v, grad in ((y, d_y), (w, d_w)):
        for at in np.ndindex(*v.shape):
            was, side = v[at], []
            for eps in (1e-3, -1e-3):
                v[at] = was + eps
                side.append((P.unpermute(y, rows, w)[0] * d_out).sum())
            v[at] = was
            want = 0.0 if np.isnan(grad[at]) else grad[at]  # a row that no slot has
            # linear in y and in w: the difference is off by roundings alone, a few 2^-52 of terms near 50, over 2e-3
            assert abs((side[0] - side[1]) / 2e-3 - want) < 1e-9


def test_quantisation_groups_by_hand():
    x = np.zeros((2, 160))
    x[0, 0], x[0, 127], x[0, 128] = 448.0, -1.0, 450.0
    x[1, 3], x[1, 130] = np.inf, np.nan
    codes, scales = P.quantize_rows(x)
    assert scales.tolist() == [[1.0, 2.0 ** 127], [2.0, 2.0 ** -126]]
    lut = F.e4m3_lut()
    assert lut[codes[0, 0]] == 448.0 and lut[codes[0, 127]] == -1.0 and lut[codes[0, 128]] == 224.0  # 225 to 224
    assert lut[codes[1, 3]] == 448.0 and lut[codes[1, 130]] == 0.0
    wc, ws = P.quantize_weights(x.reshape(1, 2, 160)[:, :1])
    assert ws.tolist() == [[[1.0, 2.0]]] and np.array_equal(wc[0, 0], codes[0])


def test_column_blocks_follow_the_segments():
    g = np.random.default_rng(1)
    x = g.standard_normal((300, 16))
    seg = [0, 130, 130, 131, 290]
    codes, scales = P.quantize_cols(x, seg)
    assert codes.shape == (128 * 5, 16) and P.padded_rows(300, 4) >= 128 * 5
    v = P.values_cols(codes, scales)
    back = np.concatenate([v[:130], v[256:257], v[384:384 + 159]])
    # half a unit of E4M3's three fraction bits, or of its smallest step at the group's scale (amax up to 448 * 2^e)
    step = np.concatenate([np.repeat(scales[:2], 128, 0)[:130], scales[2:3], np.repeat(scales[3:], 128, 0)[:159]])
    assert (np.abs(back - x[:290]) <= np.maximum(np.abs(x[:290]) * 2.0 ** -4, step * 2.0 ** -10)).all()
    for empty in (slice(130, 256), slice(257, 384), slice(384 + 159, 640)):
        assert (codes[empty] == 0).all()


@pytest.mark.parametrize("rows,E", [(0, 1), (1, 1), (128, 1), (129, 1), (5, 9), (1000, 7), (2 ** 30, 1024)])
def test_padded_rows_hold_any_counts(rows, E):
    n = K.kmoe_fp8_padded_rows(rows, E)
    assert n == P.padded_rows(rows, E) and n % 128 == 0
    # the worst counts: one row more than whole blocks for as many experts as have rows
    with_rows = min(rows, E)
    if with_rows:
        worst = [1] * with_rows
        left = rows - with_rows
        worst[0] += left
        assert sum(-(-c // 128) for c in worst) * 128 <= n


def test_products_are_each_others_gradients():
    """<d_y, x w^T> as a function of x and of w has the gradients gemm(transpose) and wgrad."""
    g = np.random.default_rng(2)
    seg = [0, 3, 3, 128]
    x, w, d_y = g.standard_normal((128, 6)), g.standard_normal((3, 4, 6)), g.standard_normal((128, 4))
    d_x = P.gemm(d_y, w, seg, transpose=True)[0]
    pad = lambda v: np.concatenate([np.pad(v[a:b], ((0, -(b - a) % 128), (0, 0))) for a, b in zip(seg, seg[1:])])  # noqa: E731
    d_w = P.wgrad(pad(d_y), pad(x), seg)[0]
    loss = lambda: (P.gemm(x, w, seg)[0] * d_y).sum()  # noqa: E731
    for v, grad, ats in ((x, d_x, [(0, 0), (2, 5), (127, 3)]), (w, d_w, [(0, 1, 2), (1, 0, 0), (2, 3, 5)])):
        for at in ats:
            was, side = v[at], []
            for eps in (1e-3, -1e-3):
                v[at] = was + eps
                side.append(loss())
            v[at] = was
            assert abs((side[0] - side[1]) / 2e-3 - grad[at]) < 1e-8  # linear: roundings of a sum near 1e3 over 2e-3


# ---------------------------------------------------------------- the C entry points


def test_the_header_and_the_binding_agree():
    hdr = open(os.path.join(ROOT, "include", "kmoe_products.h")).read()
    declared = set(re.findall(r"^\s*(?:const char\*|int|size_t)\s+(kmoe_\w+)\s*\(", hdr, re.M))
    assert declared == set(K.PRODUCT_EXPORTS)
    lib = ctypes.CDLL(K.LIB_PATH)
    for name in declared:
        assert hasattr(lib, name) and hasattr(K, name)
    for flag, value in re.findall(r"^#define (KMOE_\w+) (\d)u$", hdr, re.M):
        assert getattr(K, flag) == int(value)
    assert re.search(r"KMOE_GEMM_FP8_WORKSPACE_BYTES \(\(size_t\)%d\)" % K.GEMM_FP8_WORKSPACE_BYTES, hdr)
    assert '#include "kmoe_products.h"' in open(os.path.join(ROOT, "include", "kmoe.h")).read()


A = 4096  # an address that no call below reads: each is refused before anything is launched, or has nothing to do


def refused(name, args, status):
    got = getattr(K.lib(), name)(*args)
    assert got == status, (name, args, got)


def each(name, good, changes):
    """`good` with each (position, value, status) change on its own."""
    for at, value, status in changes:
        args = list(good)
        args[at] = value
        refused(name, args, status)


def test_refusals_of_the_sort_and_the_moves():
    n = K.kmoe_sort_workspace_size(4, 8, 2)
    assert n > 0
    for bad in ((-1, 8, 2), (4, 0, 2), (4, 1025, 2), (4, 8, 0), (4, 8, 33), (2 ** 30, 8, 2)):
        assert K.kmoe_sort_workspace_size(*bad) == 0
    each("kmoe_sort_tokens", [A, 4, 8, 2, A, A, A, A, n, None],
         [(0, None, ARG), (0, A + 2, ALIGN), (1, -1, ARG), (1, 2 ** 30, SHAPE), (2, 0, ARG), (2, 1025, ARG), (3, 0, ARG),
          (3, 33, ARG), (4, None, ARG), (4, A + 1, ALIGN), (5, None, ARG), (5, A + 2, ALIGN), (6, None, ARG),
          (6, A + 2, ALIGN), (7, None, WORKSPACE), (7, A + 128, ALIGN), (8, n - 1, WORKSPACE)])
    each("kmoe_permute", [A, A, 4, 64, 2, 0, A, None],
         [(0, None, ARG), (0, A + 8, ALIGN), (1, None, ARG), (1, A + 2, ALIGN), (2, -1, ARG), (2, 2 ** 30, SHAPE),
          (3, 0, ARG), (3, 60, SHAPE), (3, 2 ** 20 + 8, SHAPE), (4, 0, ARG), (4, 33, ARG), (5, 2, ARG), (6, None, ARG),
          (6, A + 8, ALIGN)])
    each("kmoe_unpermute", [A, A, A, 4, 64, 2, 0, A, None],
         [(0, None, ARG), (0, A + 8, ALIGN), (1, None, ARG), (1, A + 2, ALIGN), (2, A + 2, ALIGN), (3, -1, ARG),
          (4, 60, SHAPE), (4, -8, ARG), (5, 0, ARG), (6, 4, ARG), (7, None, ARG), (7, A + 4, ALIGN)])
    each("kmoe_unpermute_backward", [A, A, A, A, 4, 64, 2, 0, A, A, None],
         [(0, None, ARG), (0, A + 8, ALIGN), (1, None, ARG), (1, A + 8, ALIGN), (2, None, ARG), (3, None, ARG),
          (3, A + 2, ALIGN), (4, -1, ARG), (5, 12, SHAPE), (6, 33, ARG), (7, 4, ARG), (8, None, ARG), (8, A + 8, ALIGN),
          (9, None, ARG), (9, A + 2, ALIGN)])


def test_refusals_of_the_quantisers():
    many = K.kmoe_quantize_fp8_workspace_size(8192, 256, 16)
    assert many >= 4 * (8192 * 2 + 8192 * 16) and K.kmoe_quantize_fp8_workspace_size(100, 256, 2) == 0
    assert K.kmoe_quantize_fp8_workspace_size(8192, 100, 16) == 0
    each("kmoe_quantize_fp8", [A, 4, 64, A, 2, A, A, None, 0, None],
         [(0, None, ARG), (0, A + 8, ALIGN), (1, -1, ARG), (1, 2 ** 30, SHAPE), (2, 0, ARG), (2, 40, SHAPE),
          (2, 2 ** 20 + 16, SHAPE), (3, None, ARG), (3, A + 2, ALIGN), (4, 0, ARG), (4, 33, ARG), (5, None, ARG),
          (5, A + 8, ALIGN), (6, None, ARG), (6, A + 2, ALIGN)])
    refused("kmoe_quantize_fp8", [A, 8192, 256, A, 16, A, A, A, many - 1, None], WORKSPACE)
    each("kmoe_quantize_fp8_weights", [A, 2, 64, 64, A, A, None],
         [(0, None, ARG), (0, A + 8, ALIGN), (1, 0, ARG), (1, 1025, ARG), (2, 0, ARG), (2, 24, SHAPE), (3, 24, SHAPE),
          (4, None, ARG), (4, A + 4, ALIGN), (5, None, ARG), (5, A + 2, ALIGN)])
    each("kmoe_quantize_fp8_cols", [A, 40, 64, A, 3, A, A, None],
         [(0, None, ARG), (0, A + 8, ALIGN), (1, -1, ARG), (1, 2 ** 30 + 1, SHAPE), (2, 0, ARG), (2, 72, SHAPE),
          (3, None, ARG), (3, A + 2, ALIGN), (4, 0, ARG), (4, 1025, ARG), (5, None, ARG), (5, A + 8, ALIGN),
          (6, None, ARG), (6, A + 2, ALIGN)])
    assert K.kmoe_fp8_padded_rows(-1, 1) == -1 and K.kmoe_fp8_padded_rows(1, 0) == -1
    assert K.kmoe_fp8_padded_rows(1, 1025) == -1


def test_refusals_of_the_products():
    each("kmoe_gemm_fp8", [A, A, A, A, A, 40, 64, 32, 3, 0, A, A, 256, None],
         [(0, None, ARG), (0, A + 8, ALIGN), (1, None, ARG), (1, A + 2, ALIGN), (2, None, ARG), (2, A + 8, ALIGN),
          (3, None, ARG), (3, A + 2, ALIGN), (4, None, ARG), (4, A + 2, ALIGN), (5, -1, ARG), (6, 0, ARG), (6, 40, SHAPE),
          (7, 40, SHAPE), (7, 2 ** 20 + 16, SHAPE), (8, 0, ARG), (8, 1025, ARG), (9, 4, ARG), (10, None, ARG),
          (10, A + 8, ALIGN), (11, None, WORKSPACE), (11, A + 128, ALIGN), (12, 255, WORKSPACE)])
    # more work items than can be counted
    refused("kmoe_gemm_fp8", [A, A, A, A, None, 2 ** 30, 2 ** 20, 16, 1, 0, A, A, 256, None], SHAPE)
    each("kmoe_gemm_fp8_wgrad", [A, A, A, A, A, 256, 64, 32, 2, A, A, 256, None],
         [(0, None, ARG), (0, A + 8, ALIGN), (1, None, ARG), (1, A + 2, ALIGN), (2, None, ARG), (2, A + 8, ALIGN),
          (3, None, ARG), (4, None, ARG), (4, A + 2, ALIGN), (5, -128, ARG), (5, 200, SHAPE), (6, 40, SHAPE),
          (7, 0, ARG), (8, 0, ARG), (9, None, ARG), (9, A + 2, ALIGN), (10, None, WORKSPACE), (11, 16, WORKSPACE)])
    refused("kmoe_gemm_fp8_wgrad", [A, A, A, A, A, 256, 2 ** 20, 2 ** 20, 1024, A, A, 256, None], SHAPE)


def test_empty_batches_need_no_pointers():
    """Nothing is launched: these run without a GPU."""
    lib = K.lib()
    assert lib.kmoe_permute(None, None, 0, 64, 2, 0, None, None) == 0
    assert lib.kmoe_unpermute(None, None, None, 0, 64, 2, 0, None, None) == 0
    assert lib.kmoe_unpermute_backward(None, None, None, None, 0, 64, 2, 0, None, None, None) == 0
    assert lib.kmoe_quantize_fp8(None, 0, 64, None, 1, None, None, None, 0, None) == 0
    assert lib.kmoe_quantize_fp8_cols(None, 0, 64, None, 1, None, None, None) == 0
    assert lib.kmoe_gemm_fp8(None, None, None, None, None, 0, 64, 32, 1, 0, None, A, 256, None) == 0


# ---------------------------------------------------------------- the binding


def test_refusals_of_the_binding():
    u8, f32, i32, bf = torch.uint8, torch.float32, torch.int32, torch.bfloat16
    z = lambda d, *s: torch.zeros(*s, dtype=d)  # noqa: E731
    rows = z(i32, 4, 2)
    for call, match in (
            (lambda: K.kmoe_sort_tokens(z(torch.int64, 4, 2), 8), "topk_ids must be"),
            (lambda: K.kmoe_sort_tokens(z(i32, 8), 8), "topk_ids must be a 2-D"),
            (lambda: K.kmoe_sort_tokens(rows, 8, seg_start=z(i32, 8)), "seg_start must have shape"),
            (lambda: K.kmoe_permute(z(torch.float16, 4, 64), rows), "x must be torch.bfloat16 or"),
            (lambda: K.kmoe_permute(z(bf, 5, 64), rows), "row_of_slot must have shape"),
            (lambda: K.kmoe_permute(z(bf, 4, 128)[:, ::2], rows), "x must be contiguous"),
            (lambda: K.kmoe_permute(z(bf, 4, 64), rows, out=z(f32, 8, 64)), "out must be"),
            (lambda: K.kmoe_unpermute(z(bf, 7, 64), rows), "y must have shape"),
            (lambda: K.kmoe_unpermute(z(bf, 8, 64), rows, z(f32, 4, 3)), "topk_w must have shape"),
            (lambda: K.kmoe_unpermute(z(bf, 8, 64), rows, out_dtype=torch.float16), "out_dtype must be"),
            (lambda: K.kmoe_unpermute_backward(z(bf, 4, 64), z(bf, 8, 64), rows, z(bf, 4, 2)), "topk_w must be"),
            (lambda: K.kmoe_unpermute_backward(z(bf, 4, 64), z(bf, 8, 64), rows, None, d_y=z(f32, 8, 64)), "d_y must be"),
            (lambda: K.kmoe_quantize_fp8(z(f32, 4, 64)), "x must be torch.bfloat16"),
            (lambda: K.kmoe_quantize_fp8(z(bf, 4, 144), scales=z(f32, 4, 2)), "scales must have shape"),
            (lambda: K.kmoe_quantize_fp8_weights(z(bf, 4)), r"\[E, N, K\]"),
            (lambda: K.kmoe_quantize_fp8_cols(z(bf, 4, 64), seg_start=z(i32, 1)), "seg_start must be"),
            (lambda: K.kmoe_gemm_fp8(z(u8, 4, 64), z(f32, 1, 4), z(u8, 2, 32, 64), z(f32, 2, 1, 1)), "holds 2 experts"),
            (lambda: K.kmoe_gemm_fp8(z(u8, 4, 64), z(f32, 4, 1), z(u8, 32, 64), z(f32, 1, 1)), "x_scales must have shape"),
            (lambda: K.kmoe_gemm_fp8(z(u8, 4, 64), z(f32, 1, 4), z(u8, 32, 64), z(f32, 1, 1), transpose=True),
             "x must have shape"),
            (lambda: K.kmoe_gemm_fp8(z(u8, 4, 64), z(f32, 1, 4), z(u8, 32, 64), z(f32, 1, 1), workspace=z(u8, 100)),
             "workspace holds 100 bytes"),
            (lambda: K.kmoe_gemm_fp8_wgrad(z(u8, 128, 64), z(f32, 1, 64), z(u8, 128, 32), z(f32, 2, 32)),
             "x_scales must have shape"),
            (lambda: K.kmoe_gemm_fp8(z(u8, 4, 64), z(f32, 1, 4), z(u8, 32, 64), z(f32, 1, 1)), "must be a CUDA tensor")):
        with pytest.raises(ValueError, match=match):
            call()
