"""GPU checks of the block-scaled products with scales of any size.

Tolerances are test_gpu_products'; besides, a result below 2^-126 has 2^-149 for
its last place (bf16: 2^-133), and where the product of a block's two scales is
below 2^-126 that product is off by up to 2^-150 and the block, whose sum is at
most 128 * 448^2 < 2^24.7, by 2^-125."""
import numpy as np
import pytest
import torch

from oracle import products as P
from tests.test_gpu_products import BF, F32, K, f64, no_error, product_tolerance, random_codes  # noqa: F401 (K: a fixture)

pytestmark = pytest.mark.gpu
TOP = float(np.finfo(np.float32).max)


def run(K, x, xs, w, ws, transpose, to):  # noqa: F811
    out, work = K.kmoe_gemm_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), transpose=transpose, out_dtype=to)
    no_error(K, work)
    return f64(out)


def check(K, x, xs, w, ws, transpose, low=False):  # noqa: F811
    """`low`: some scales' products are below 2^-126."""
    _, N, Kd = w.shape
    n = N if transpose else Kd
    ref, mag = P.gemm(P.values_rows(x.numpy(), xs.numpy()), P.values_weights(w.numpy(), ws.numpy()), [0, x.shape[0]],
                      transpose)
    sure = mag < TOP / 2  # no sum of some of the terms overflows, nor rounds to an infinity
    blocks = -(-n // 128)
    for to in (F32, BF):
        got = run(K, x, xs, w, ws, transpose, to)
        assert (got[mag == 0] == 0).all()
        tol = product_tolerance(ref, mag, n, to) + (blocks + 1) * 2.0 ** -149 + (2.0 ** -134 if to is BF else 0.0)
        tol = tol + (blocks * 2.0 ** -125 * (1 + 2.0 ** -7) if low else 0.0)
        bad = sure & ~(np.abs(got - ref) <= tol)
        assert not bad.any(), (to, bad.sum(), np.argwhere(bad)[:3], got[bad][:3], ref[bad][:3], tol[bad][:3])
    return ref, mag


# both kernels, whole and partial tiles of features, items alone and shared by clusters
SHAPES = [(30, 272, 400), (1, 256, 4096), (20, 128, 1024), (300, 272, 400), (129, 272, 2176), (64, 400, 272), (40, 16, 128)]


def inputs(M, N, Kd, transpose, rows, cols):
    """Codes, row 0 zeros, with the scales `rows` by row and `cols` by block of features, the same over the sum's blocks."""
    wide = N if transpose else Kd
    x, w = random_codes(M, M, wide), random_codes(N, 1, N, Kd)
    if M > 1:
        x[0] = 0
    nb, kb = -(-N // 128), -(-Kd // 128)
    xs = torch.from_numpy(np.resize(np.array(rows, np.float32), M))[None].repeat(-(-wide // 128), 1).contiguous()
    c = torch.from_numpy(np.resize(np.array(cols, np.float32), kb if transpose else nb))
    ws = c[None].repeat(nb, 1) if transpose else c[:, None].repeat(1, kb)
    return x, xs, w, ws[None].contiguous()


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("M,N,Kd", SHAPES)
def test_scales_far_from_one(K, M, N, Kd, transpose):  # noqa: F811
    """Scales at the ends of fp32 whose product is a normal number."""
    for rows, cols in (([2.0 ** 127, 3e30, -2.0 ** 126, 0.0], [1.2345e-38, -3e-20, 2.0 ** -126, 0.0]),
                       ([2.0 ** -126, -1.5 * 2.0 ** -125, 0.0], [1.0, 2.0 ** 127, -3.7, 1e20]),
                       ([2.0 ** -149, -2.0 ** -140, 0.0], [2.0 ** 30, 2.0 ** 127, 1e15])):
        for shift in range(len(cols)):
            check(K, *inputs(M, N, Kd, transpose, rows, np.roll(cols, -shift)), transpose)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("M,N,Kd", SHAPES)
def test_products_of_scales_below_the_range(K, M, N, Kd, transpose):  # noqa: F811
    rows, cols = [2.0 ** -126, 1e-30, -2.0 ** -140, 1.0, 2.0 ** -149], [1.2345e-4, 1e-20, 2.0 ** -126, -0.37]
    for shift in range(len(cols)):
        check(K, *inputs(M, N, Kd, transpose, rows, np.roll(cols, -shift)), transpose, low=True)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("M,N,Kd", SHAPES)
def test_blocks_of_different_sizes(K, M, N, Kd, transpose):  # noqa: F811
    """Blocks in and below the range within a sum."""
    wide = N if transpose else Kd
    g = np.random.default_rng(M + N)
    x, w = random_codes(M, M, wide), random_codes(N, 1, N, Kd)
    xs = np.exp2(g.integers(-126, -60, (-(-wide // 128), M))) * g.uniform(1, 2)
    ws = np.exp2(g.integers(-40, -5, (1, -(-N // 128), -(-Kd // 128)))) * g.uniform(1, 2)
    check(K, x, torch.from_numpy(xs.astype(np.float32)), w, torch.from_numpy(ws.astype(np.float32)), transpose, low=True)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("M,N,Kd", SHAPES)
def test_products_of_scales_beyond_the_range(K, M, N, Kd, transpose):  # noqa: F811
    """Infinite or NaN in their rows, and nothing changed in the others'."""
    x, xs, w, ws = inputs(M, N, Kd, transpose, [1.0], [4.0])
    before = run(K, x, xs, w, ws, transpose, F32)
    at = M - 1
    xs[-1, at] = 2.0 ** 127
    after = run(K, x, xs, w, ws, transpose, F32)
    assert not np.isfinite(after[at]).any()
    keep = np.arange(M) != at
    assert (after[keep] == before[keep]).all()


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("M", [20, 300])
def test_rows_that_the_quantiser_made(K, M, transpose):  # noqa: F811
    """Rows of tiny values, of zeros and with an infinity, by way of kmoe_quantize_fp8."""
    N, Kd = 272, 400
    wide = N if transpose else Kd
    g = torch.Generator().manual_seed(M)
    x = torch.randn(M, wide, generator=g)
    x[3] *= 1e-36
    x[7] *= 1e-38
    x[9, :128] = 0
    x[10] = 0
    x[11, 5] = float("inf")
    xc, xs = (t.cpu() for t in K.kmoe_quantize_fp8(x.to(BF).cuda()))
    assert xs[0, 3] == 2.0 ** -126 and xs[0, 10] == 2.0 ** -126 and xs[0, 11] == 2.0 ** 127
    w = random_codes(5, 1, N, Kd)
    scales = torch.full((1, -(-N // 128), -(-Kd // 128)), 1.2345e-4)
    ref, mag = check(K, xc, xs, w, scales, transpose, low=True)
    assert (mag[10] == 0).all() and (mag[11] > 1e30).any()
