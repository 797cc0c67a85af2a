"""GPU checks that no part of a long sum is lost in the block-scaled products.

Whole numbers: codes of 0, 1 and 2 in size with power-of-two scales, whose
products and partial sums are whole numbers below 2^24 (or such times one power
of two): every fp32 sum of them is exact, so equality shows every block.

Norms of random sums.  Additions that round to nearest are each off by at most
2^-24 of a partial sum, whose size in the 2-norm over the outputs is at most the
whole's; errors of either sign add in squares: sqrt(n) * 2^-24 for n additions.
A product has one addition a block of 128, one rounding of its factor, and four
steps of the tensor core inside, each of which may drop a last place, 2^-23 of
the block (its blocks are independent: 4 * 2^-23 = 2^-21 bounds them).  The
weights' gradient has 32 such steps in a run of 1024 rows, whose errors have the
sum's sign: the i-th is half a last place on average, 2^-24, of a partial sum of
sqrt(i / 32) of the run's size, 21.8 * 2^-24 together; and an addition a run."""
import numpy as np
import pytest
import torch

from oracle import formats as F
from oracle import products as P
from tests.test_gpu_products import (BF, F32, K, f64, no_error, product_inputs, randn, segments)  # noqa: F401 (K: a fixture)

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


def whole_numbers(seed, *shape):
    return np.random.default_rng(seed).integers(-2, 3, shape).astype(np.float64)


def codes(v):
    return torch.from_numpy(F.round_to_code(v, "e4m3"))


def seg_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


# long sums, every cluster size, several items a CTA, uneven experts
WHOLE = [(1, 32, 131072, None), (2, 131072, 144, None), (40, 32, 65552, None), (130, 65552, 48, None), (5, 2048, 1040, None),
         (32, 640, 4112, None), (64, 1024, 4096, None), (129, 272, 2176, None), (2600, 4112, 144, None),
         (512, 272, 1040, [400, 0, 1, 7, 33] + [1] * 59 + [12]), (1500, 144, 528, [1000, 129, 0, 371])]


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("M,N,Kd,counts", WHOLE)
def test_every_block_of_a_product_counts(K, M, N, Kd, counts, transpose):  # noqa: F811
    E = 1 if counts is None else len(counts)
    seg = seg_of([M] if counts is None else counts)
    assert seg[-1] == M
    wide, n = (N, N) if transpose else (Kd, Kd)
    x, w = whole_numbers(M, M, wide), whole_numbers(N + 1, E, N, Kd)
    b = np.arange(-(-wide // 128))
    xs = np.exp2((b[:, None] + np.arange(M)) % 3)  # 1, 2, 4
    nb, kb = np.arange(-(-N // 128)), np.arange(-(-Kd // 128))
    ws = np.exp2(-((nb[:, None] + 2 * kb) % 2))[None].repeat(E, 0)  # 1, 1/2
    assert n * 4 * 4 * 2 <= 2 ** 24  # twice the sums are whole numbers
    ref, _ = P.gemm(x * np.repeat(xs.T, 128, 1)[:, :wide], w * np.repeat(np.repeat(ws, 128, 1), 128, 2)[:, :N, :Kd], seg, transpose)
    out, work = K.kmoe_gemm_fp8(codes(x).cuda(), torch.from_numpy(xs.astype(np.float32)).cuda(), codes(w).cuda(),
                                torch.from_numpy(ws.astype(np.float32)).cuda(),
                                None if E == 1 else torch.from_numpy(seg).cuda(), transpose=transpose, out_dtype=F32)
    no_error(K, work)
    assert np.array_equal(f64(out), ref)


@pytest.mark.parametrize("rows,N,Kd,counts", [(65536, 144, 128, None), (5000, 272, 400, None), (1, 16, 16, None),
                                              (3000, 240, 272, [1025, 0, 1, 1024, 127, 823])])
def test_every_block_of_the_weights_gradient_counts(K, rows, N, Kd, counts):  # noqa: F811
    E = 1 if counts is None else len(counts)
    seg = seg_of([rows] if counts is None else counts)
    dy, x = whole_numbers(rows, rows, N), whole_numbers(rows + 1, rows, Kd)
    dy *= np.exp2(np.arange(rows) // 100 % 4)[:, None]  # up to 16: blocks of different scales
    assert rows * 16 * 2 <= 2 ** 24
    sg = None if E == 1 else torch.from_numpy(seg).cuda()
    qd, qx = (K.kmoe_quantize_fp8_cols(torch.from_numpy(v).to(BF).cuda(), sg) for v in (dy, x))
    dw, work = K.kmoe_gemm_fp8_wgrad(*qd, *qx, seg_start=sg)
    no_error(K, work)
    ref = np.stack([dy[a:b].T @ x[a:b] for a, b in zip(seg[:-1], seg[1:])])
    assert np.array_equal(f64(dw), ref)


def off(got, ref):
    return np.linalg.norm(f64(got) - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("M,N,Kd", [(1, 32, 131072), (2, 131072, 144), (40, 32, 65552), (130, 65552, 48), (200, 3600, 2064)])
def test_long_products_in_the_norm(K, M, N, Kd, transpose):  # noqa: F811
    x, xs, w, ws, seg = product_inputs(M, N, Kd, 1, transpose)
    ref, _ = P.gemm(P.values_rows(x.numpy(), xs.numpy()), P.values_weights(w.numpy(), ws.numpy()), seg, transpose)
    out, work = K.kmoe_gemm_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), transpose=transpose, out_dtype=F32)
    no_error(K, work)
    blocks = -(-(N if transpose else Kd) // 128)
    assert off(out, ref) <= (np.sqrt(blocks) + 1) * U32 + 2.0 ** -21


@pytest.mark.parametrize("rows", [1000, 16000, 65536])
def test_weights_gradient_in_the_norm(K, rows):  # noqa: F811
    dy, x = randn(1, rows, 144).to(BF).cuda(), randn(2, rows, 128).to(BF).cuda()
    qd, qx = K.kmoe_quantize_fp8_cols(dy), K.kmoe_quantize_fp8_cols(x)
    dw, work = K.kmoe_gemm_fp8_wgrad(*qd, *qx)
    no_error(K, work)
    ref, _ = P.wgrad(*(P.values_cols(c.cpu().numpy(), s.cpu().numpy()) for c, s in (qd, qx)), [0, rows])
    # 65536 rows: 1.8e-6; all of them in the tensor core's accumulator were 7e-6 off
    assert off(dw, ref) <= (21.8 + np.sqrt(-(-rows // 1024))) * U32


@pytest.mark.parametrize("rows,E", [(300, 1), (900, 3)])
def test_weights_gradient_of_very_large_and_small_rows(K, rows, E):  # noqa: F811
    """Scales at the ends of fp32, whose products are not."""
    N, Kd = 144, 272
    seg = segments(rows, rows, E)
    sg = None if E == 1 else torch.from_numpy(seg).cuda()
    for a, b in ((2.0 ** -118, 2.0 ** 118), (2.0 ** 118, 2.0 ** -118), (2.0 ** -60, 2.0 ** -40), (2.0 ** 60, 2.0 ** 40)):
        dy, x = (randn(1, rows, N) * a).to(BF).cuda(), (randn(2, rows, Kd) * b).to(BF).cuda()
        qd, qx = K.kmoe_quantize_fp8_cols(dy, sg), K.kmoe_quantize_fp8_cols(x, sg)
        dw, work = K.kmoe_gemm_fp8_wgrad(*qd, *qx, seg_start=sg)
        no_error(K, work)
        n = sum(-(-(q - p) // 128) * 128 for p, q in zip(seg[:-1], seg[1:]))
        ref, mag = P.wgrad(*(P.values_cols(c.cpu().numpy()[:n], s.cpu().numpy()[:n // 128]) for c, s in (qd, qx)), seg)
        assert off(dw, ref) <= (21.8 + np.sqrt(-(-rows // 1024))) * U32
