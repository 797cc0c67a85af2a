"""GPU checks of the sort by expert and back and of the block-scaled E4M3
products against the float64 definitions of oracle.products.

Tolerances.  Sorts, moves and quantisation are exact.  A sum of n fp32 terms is
off by at most n * 2^-24 of the sum of the absolute terms when every addition
rounds to nearest, and n * 2^-23 when it truncates; a product's terms are the
exact products of two 8-bit values in blocks of 128, each block's sum scaled
(two roundings) and added to the others.  A value stored in bf16 is off by at
most half a unit in the last place, 2^-8 of it."""
import numpy as np
import pytest
import torch

from oracle import formats as F
from oracle import products as P

pytestmark = pytest.mark.gpu
U32, UBF = 2.0 ** -24, 2.0 ** -8
BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
E4M3 = F.e4m3_lut()


@pytest.fixture(scope="module")
def K():
    import mxfp8_mxfp4_moe_gb300 as K
    assert K.kmoe_check_device(0) == 0
    return K


def randn(seed, *shape):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32))


def f64(t):
    return t.detach().double().cpu().numpy()


def within(got, ref, tol, what):
    g = f64(got)
    assert g.shape == ref.shape
    bad = ~((np.abs(g - ref) <= tol) | (np.isnan(ref) & np.isnan(g)))  # NaN is off unless it is meant
    i = np.unravel_index(np.argmax(bad), ref.shape) if ref.size else None
    assert not bad.any(), f"{what}: {bad.sum()} of {ref.size} off, at {i}: {g[i]!r} against {ref[i]!r}, {tol[i]!r} allowed"


def no_error(K, ws):
    st, word = K.kmoe_device_error(ws)
    assert st == 0, hex(word)


def routing(seed, T, E, k, masked=0.0):
    """ids [T, k]; some experts popular, some never chosen, `masked` of the slots none."""
    g = np.random.default_rng(seed)
    p = np.exp(g.standard_normal(E)) * (g.random(E) < 0.8)
    p = p / p.sum() if p.sum() > 0 else np.full(E, 1.0 / E)
    ids = g.choice(E, size=(T, k), p=p).astype(np.int32)
    ids[g.random((T, k)) < masked] = -1
    return ids


# ---------------------------------------------------------------- sort, permute, unpermute

SORTS = [(1, 1, 1), (1, 8, 4), (16, 896, 16), (64, 64, 16), (65, 7, 16), (1024, 3, 1), (1025, 1024, 1), (500, 31, 32),
         (3000, 897, 7), (2048, 2, 1)]


@pytest.mark.parametrize("T,E,k", SORTS)
def test_sort(K, T, E, k):
    ids = routing(T + E, T, E, k, 0.1)
    if T > 2:
        ids[T // 2, 0], ids[T // 3, 0] = E, 2 ** 31 - 1  # no experts
    row, slot, seg = K.kmoe_sort_tokens(torch.from_numpy(ids).cuda(), E)
    ref = P.sort_tokens(ids, E)
    for got, want in zip((row, slot, seg), ref):
        assert np.array_equal(got.cpu().numpy(), want)


def test_sort_masked_batches(K):
    for T, E, k in ((5, 4, 3), (2000, 100, 4)):
        row, slot, seg = K.kmoe_sort_tokens(torch.full((T, k), -1, dtype=I32, device="cuda"), E)
        assert (row == -1).all() and (slot == -1).all() and (seg == 0).all()
    row, slot, seg = K.kmoe_sort_tokens(torch.empty(0, 4, dtype=I32, device="cuda"), 9)
    assert row.shape == (0, 4) and slot.shape == (0,) and (seg == 0).all()


def sorted_rows(T, E, k, masked=0.1):
    ids = routing(3 * T + k, T, E, k, masked)
    row, slot, seg = P.sort_tokens(ids, E)
    return ids, row, seg


MOVES = [(1, 8, 1, 1), (1, 7168, 8, 4), (17, 5000, 64, 8), (129, 3584, 64, 8), (640, 264, 9, 32), (700, 4104, 33, 3)]


@pytest.mark.parametrize("ty", [BF, F32])
@pytest.mark.parametrize("T,H,E,k", MOVES)
def test_permute(K, T, H, E, k, ty):
    _, row, seg = sorted_rows(T, E, k)
    x = randn(T, T, H).to(ty).cuda()
    x[0, 0] = float("nan")
    out = torch.full((T * k, H), 7.0, dtype=ty, device="cuda")
    K.kmoe_permute(x, torch.from_numpy(row).cuda(), out=out)
    want = torch.full((T * k, H), 7.0, dtype=ty)
    for t, j in np.argwhere(row >= 0):
        want[row[t, j]] = x[t].cpu()
    assert torch.equal(out.cpu().nan_to_num(-9.0), want.nan_to_num(-9.0))


@pytest.mark.parametrize("ty,to", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("T,H,E,k", MOVES)
def test_unpermute(K, T, H, E, k, ty, to):
    _, row, seg = sorted_rows(T, E, k)
    y = randn(T, T * k, H).to(ty).cuda()
    y[seg[E]:] = float("nan")  # rows that no slot has are not read
    w = randn(T + 1, T, k).cuda()
    for weights in (w, None):
        out = K.kmoe_unpermute(y, torch.from_numpy(row).cuda(), weights, out_dtype=to)
        ref, mag = P.unpermute(f64(y), row, None if weights is None else f64(w))
        tol = k * U32 * mag + (UBF * np.abs(ref) + UBF * k * U32 * mag if to is BF else 0.0)
        within(out, ref, tol, "unpermute")


@pytest.mark.parametrize("tg,ty", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("T,H,E,k", MOVES + [(160, 520, 5, 32)])
def test_unpermute_backward(K, T, H, E, k, tg, ty):
    _, row, seg = sorted_rows(T, E, k)
    y = randn(T, T * k, H).to(ty).cuda()
    y[seg[E]:] = float("nan")
    w, g = randn(T + 1, T, k).cuda(), randn(T + 2, T, H).to(tg).cuda()
    d_y0 = torch.full_like(y, float("nan"))
    d_y, d_w = K.kmoe_unpermute_backward(g, y, torch.from_numpy(row).cuda(), w, d_y=d_y0)
    ref_y, ref_w, mag = P.unpermute_backward(f64(g), f64(y), row, f64(w))
    within(d_y, ref_y, (U32 if ty is F32 else UBF + 2 * U32) * np.abs(ref_y), "d_y")
    within(d_w, ref_w, (H + 1) * U32 * mag, "d_w")
    # in place
    same, d_w2 = K.kmoe_unpermute_backward(g, y, torch.from_numpy(row).cuda(), w, d_y=y)
    assert same is y and torch.equal(d_w2, d_w) and torch.equal(y[:seg[E]], d_y[:seg[E]])


def test_unpermute_gradient_against_differences(K):
    """<d_out, unpermute(y, w)> moves by <d_y, dy> + <d_w, dw> (fp32 rows: linear in each)."""
    T, H, E, k = 9, 40, 6, 4
    _, row, seg = sorted_rows(T, E, k, 0.2)
    r = torch.from_numpy(row).cuda()
    y, w, g = randn(1, T * k, H).cuda(), randn(2, T, k).cuda(), randn(3, T, H).cuda()
    dy, dw = randn(4, T * k, H).cuda(), randn(5, T, k).cuda()
    d_y, d_w = K.kmoe_unpermute_backward(g, y, r, w, d_y=torch.zeros_like(y))

    def loss(y, w):
        return float((K.kmoe_unpermute(y, r, w, out_dtype=F32).double() * g.double()).sum())

    live = torch.from_numpy(row >= 0).cuda()
    for grad, fwd, bwd in (((d_y.double() * dy).sum(), loss(y + dy, w), loss(y - dy, w)),
                           ((d_w.double() * dw)[live].sum(), loss(y, w + dw), loss(y, w - dw))):
        # both sides are sums of at most T*k*H terms of size about 4, off by a few roundings each
        assert abs((fwd - bwd) / 2 - float(grad)) <= T * k * H * 8 * 8 * U32


def test_moves_are_each_others_gradients(K):
    """kmoe_unpermute without weights is kmoe_permute's gradient."""
    T, H, E, k = 37, 96, 11, 5
    _, row, seg = sorted_rows(T, E, k)
    r = torch.from_numpy(row).cuda()
    x, g = randn(1, T, H).cuda(), randn(2, T * k, H).cuda()
    xp = K.kmoe_permute(x, r, out=torch.zeros(T * k, H, device="cuda"))
    dx = K.kmoe_unpermute(g, r, out_dtype=F32)
    n = int(seg[E])
    a, b = (xp[:n].double() * g[:n].double()).sum(), (x.double() * dx.double()).sum()
    # dx is off by at most k roundings of sums of k terms, |g|, |x| below 6 in size
    assert abs(float(a - b)) <= T * H * 6 * k * 6 * k * U32


def test_moves_past_2_31_elements(K):
    T, H, k = 9500, 7168, 32  # T * k * H > 2^31
    row = torch.arange(T * k, dtype=I32, device="cuda").view(T, k)
    x = (torch.arange(T, device="cuda") % 251).to(BF)[:, None].expand(T, H).contiguous()
    xp = K.kmoe_permute(x, row)
    assert torch.equal(xp.view(T, k, H)[-1], x[-1].expand(k, H)) and torch.equal(xp.view(T, k, H)[::997, 3], x[::997])
    out = K.kmoe_unpermute(xp, row, torch.full((T, k), 1.0 / k, device="cuda"))
    assert torch.equal(out, x)
    d_y, d_w = K.kmoe_unpermute_backward(out, xp, row, torch.ones(T, k, device="cuda"), d_y=xp)
    assert torch.equal(d_y.view(T, k, H)[-1], x[-1].expand(k, H))
    assert torch.allclose(d_w[-1], (x[-1].float() ** 2).sum().expand(k))


# ---------------------------------------------------------------- quantisers


def special(seed, rows, cols):
    """Values of many sizes, whole groups of zeros, infinities, NaN, ties and scales' borders."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, cols)) * np.exp2(g.integers(-30, 30, (rows, 1)))
    x = torch.from_numpy(x.astype(np.float32)).to(BF)
    flat = x.view(-1)
    n = flat.numel()
    for i, v in enumerate([float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 448.0, 3.3e38, 1e-40, 2.0 ** -126,
                           449.0, 1.0625, 1.1875]):
        flat[(i * 977 + 5) % n] = v
    if rows > 1:
        x[1] = 0.0
    if rows > 2:
        x[2, : cols // 2] = float("nan")
    return x


def same(got, ref, what):
    got = got.cpu().numpy()
    assert got.shape == ref.shape
    bad = got != ref
    assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])


@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 7168), (3, 128), (9, 144), (33, 528), (130, 2064)])
def test_quantize_rows(K, rows, cols):
    x = special(rows, rows, cols)
    codes, scales = K.kmoe_quantize_fp8(x.cuda())
    ref_c, ref_s = P.quantize_rows(f64(x))
    same(codes, ref_c, "codes")
    same(scales.double(), ref_s, "scales")


# the last two have rows enough for the scales' own pass, of one and of two 64-group chunks
@pytest.mark.parametrize("T,cols,E,k", [(1, 16, 1, 1), (5, 7168, 8, 4), (33, 528, 7, 3), (400, 144, 9, 2),
                                        (4100, 144, 40, 16), (2048, 8400, 40, 32)])
def test_quantize_into_sorted_rows(K, T, cols, E, k):
    x = special(T, T, cols)
    _, row, seg = sorted_rows(T, E, k)
    codes = torch.full((T * k, cols), 99, dtype=U8, device="cuda")
    scales = torch.full((-(-cols // 128), T * k), -3.0, device="cuda")
    K.kmoe_quantize_fp8(x.cuda(), torch.from_numpy(row).cuda(), codes=codes, scales=scales)
    assert (K.kmoe_quantize_fp8_workspace_size(T, cols, k) > 0) == (T >= 2048)
    few = slice(None) if T < 2048 else np.r_[0:40, T - 40:T]  # the oracle's loops are slow
    ref_c, ref_s = P.quantize_rows(f64(x)[few])
    plain_c, plain_s = K.kmoe_quantize_fp8(x.cuda())  # checked row by row in the test above, and here where `few` says
    same(plain_c[few], ref_c, "codes by token")
    same(plain_s.double()[:, few], ref_s, "scales by token")
    want_c, want_s = np.full((T * k, cols), 99, np.uint8), np.full(scales.shape, -3.0)
    plain_c, plain_s = plain_c.cpu().numpy(), f64(plain_s)
    for t, j in np.argwhere(row >= 0):
        want_c[row[t, j]], want_s[:, row[t, j]] = plain_c[t], plain_s[:, t]
    same(codes, want_c, "codes")
    same(scales.double(), want_s, "scales")


@pytest.mark.parametrize("E,N,Kd", [(1, 16, 16), (1, 128, 256), (3, 144, 400), (2, 528, 128)])
def test_quantize_weights(K, E, N, Kd):
    w = special(E + N, E * N, Kd).view(E, N, Kd)
    codes, scales = K.kmoe_quantize_fp8_weights(w.cuda())
    ref_c, ref_s = P.quantize_weights(f64(w))
    same(codes, ref_c, "codes")
    same(scales.double(), ref_s, "scales")
    if E == 1:
        c2, s2 = K.kmoe_quantize_fp8_weights(w[0].cuda())
        assert torch.equal(c2, codes[0]) and torch.equal(s2, scales[0])


def segments(seed, rows, E, behind=0):
    """seg_start of E experts over rows - behind rows, some experts without any."""
    g = np.random.default_rng(seed)
    cuts = np.sort(g.integers(0, rows - behind + 1, E - 1))
    if E > 3:
        cuts[1] = cuts[0]
    return np.concatenate([[0], cuts, [rows - behind]]).astype(np.int32)


@pytest.mark.parametrize("rows,cols,E", [(1, 16, 1), (128, 144, 1), (300, 272, 1), (300, 144, 4), (77, 400, 100),
                                         (1000, 128, 3)])
def test_quantize_cols(K, rows, cols, E):
    x = special(rows, rows, cols)
    seg = segments(rows, rows, E, behind=7 if rows > 20 and E > 1 else 0)
    P_ = K.kmoe_fp8_padded_rows(rows, E)
    assert P_ == P.padded_rows(rows, E)
    codes = torch.full((P_, cols), 99, dtype=U8, device="cuda")
    scales = torch.full((P_ // 128, cols), -3.0, device="cuda")
    K.kmoe_quantize_fp8_cols(x.cuda(), None if E == 1 else torch.from_numpy(seg).cuda(), codes=codes, scales=scales)
    ref_c, ref_s = P.quantize_cols(f64(x), seg)
    n = ref_c.shape[0]
    assert n <= P_
    same(codes[:n], ref_c, "codes")
    same(scales[:n // 128].double(), ref_s, "scales")
    assert (codes[n:] == 99).all() and (scales[n // 128:] == -3.0).all()


# ---------------------------------------------------------------- products


def random_codes(seed, *shape):
    """E4M3 codes of every size but NaN, mostly near the middle of the range."""
    v = np.random.default_rng(seed).standard_normal(shape) * 20.0
    return torch.from_numpy(F.round_to_code(v, "e4m3"))


def random_scales(seed, *shape):
    return torch.from_numpy(np.exp(np.random.default_rng(seed).standard_normal(shape)).astype(np.float32) * 1e-3)


def product_inputs(M, N, Kd, E, transpose, behind=0):
    wide = N if transpose else Kd
    x, xs = random_codes(M, M, wide), random_scales(M + 1, -(-wide // 128), M)
    w, ws = random_codes(N, E, N, Kd), random_scales(N + 1, E, -(-N // 128), -(-Kd // 128))
    seg = segments(M + E, M, E, behind)
    return x, xs, w, ws, seg


def product_tolerance(ref, mag, n, to):
    acc = (n + 4) * 2 * U32 * mag  # truncating additions
    return acc + (UBF * (np.abs(ref) + acc) if to is BF else 0.0)


PRODUCTS = [(1, 16, 16, 1), (1, 128, 128, 1), (1, 528, 7168, 1), (16, 144, 144, 1), (17, 272, 400, 1), (32, 128, 1024, 1),
            (33, 256, 256, 1), (128, 640, 272, 1), (129, 128, 512, 1), (257, 400, 384, 1), (600, 144, 640, 1),
            (1000, 1040, 256, 1), (1, 144, 144, 5), (40, 272, 400, 8), (200, 144, 528, 3), (333, 256, 128, 64),
            (700, 128, 272, 2), (1500, 400, 144, 5), (3, 16, 32, 1000),
            # shared by clusters of 2, 4 and 8; several items a CTA; blocks that leave a cluster's last CTA fewer
            (5, 2048, 1040, 1), (32, 640, 4112, 1), (20, 4112, 528, 1), (64, 1024, 4096, 1), (200, 3600, 2064, 1),
            (129, 272, 2176, 1), (2600, 4112, 144, 1), (70, 6160, 144, 40), (4000, 2064, 272, 9)]


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("M,N,Kd,E", PRODUCTS)
def test_gemm(K, M, N, Kd, E, transpose):
    behind = M // 8 if E > 1 else 0
    x, xs, w, ws, seg = product_inputs(M, N, Kd, E, transpose, behind)
    ref, mag = P.gemm(P.values_rows(x.numpy(), xs.numpy()), P.values_weights(w.numpy(), ws.numpy()), seg, transpose)
    for to in (BF, F32):
        out = torch.full(ref.shape, float("nan"), dtype=to, device="cuda")
        _, work = K.kmoe_gemm_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(),
                                  None if E == 1 else torch.from_numpy(seg).cuda(), transpose=transpose, out=out)
        no_error(K, work)
        n = N if transpose else Kd
        within(out, ref, product_tolerance(ref, mag, n, to), f"{to}")


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("M,N,Kd", [(1, 32, 131072), (2, 131072, 144), (40, 32, 65552), (130, 65552, 48)])
def test_long_products(K, M, N, Kd, transpose):
    test_gemm(K, M, N, Kd, 1, transpose)


@pytest.mark.parametrize("rows,N,Kd,E", [(1, 16, 16, 1), (128, 128, 128, 1), (300, 272, 144, 1), (1000, 144, 400, 1),
                                         (129, 528, 128, 1), (300, 144, 272, 4), (77, 16, 144, 100), (900, 384, 256, 3)])
def test_wgrad(K, rows, N, Kd, E):
    seg = segments(rows, rows, E, behind=7 if rows > 20 and E > 1 else 0)
    sg = None if E == 1 else torch.from_numpy(seg).cuda()
    dy, x = randn(1, rows, N).to(BF).cuda() * 1e-2, randn(2, rows, Kd).to(BF).cuda()
    x[seg[-1]:] = float("nan")
    qd, qx = K.kmoe_quantize_fp8_cols(dy, sg), K.kmoe_quantize_fp8_cols(x, sg)
    dw = torch.full((E, N, Kd), float("nan"), device="cuda")
    _, work = K.kmoe_gemm_fp8_wgrad(*qd, *qx, seg_start=sg, dw=dw)
    no_error(K, work)
    n = sum(-(-(b - a) // 128) * 128 for a, b in zip(seg[:-1], seg[1:]))
    vd, vx = (P.values_cols(c.cpu().numpy()[:n], s.cpu().numpy()[:n // 128]) for c, s in (qd, qx))
    ref, mag = P.wgrad(vd, vx, seg)
    within(dw, ref, product_tolerance(ref, mag, rows + 128, F32), "dw")


def test_empty_batches(K):
    w, ws = random_codes(1, 2, 128, 256).cuda(), random_scales(2, 2, 1, 2).cuda()
    seg = torch.zeros(3, dtype=I32, device="cuda")
    e = lambda *s, dtype=U8: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    out, _ = K.kmoe_gemm_fp8(e(0, 256), e(2, 0, dtype=F32), w, ws, seg)
    assert out.shape == (0, 128)
    # rows, but none of an expert's
    x, xs = random_codes(3, 40, 256).cuda(), random_scales(4, 2, 40).cuda()
    out = torch.full((40, 128), 3.0, dtype=BF, device="cuda")
    _, work = K.kmoe_gemm_fp8(x, xs, w, ws, seg, out=out)
    no_error(K, work)
    assert (out == 3.0).all()
    for rows in (0, 300):
        q = [K.kmoe_quantize_fp8_cols(torch.ones(rows, c, dtype=BF, device="cuda"), seg) for c in (128, 256)]
        dw = torch.full((2, 128, 256), 5.0, device="cuda")
        _, work = K.kmoe_gemm_fp8_wgrad(*q[0], *q[1], seg_start=seg, dw=dw)
        no_error(K, work)
        assert (dw == 0).all()


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("M", [20, 300])
def test_nan_codes_stay_in_their_row(K, M, transpose):
    N, Kd = 272, 400
    x, xs, w, ws, seg = product_inputs(M, N, Kd, 1, transpose)
    args = [t.cuda() for t in (x, xs, w, ws)]
    clean, _ = K.kmoe_gemm_fp8(*args, transpose=transpose, out_dtype=F32)
    args[0][7, 5] = 0x7F
    args[1][1, 11] = float("inf")
    out, _ = K.kmoe_gemm_fp8(*args, transpose=transpose, out_dtype=F32)
    assert torch.isnan(out[7]).all() and not torch.isfinite(out[11]).any()
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[[7, 11]] = False
    assert torch.equal(out[keep], clean[keep])


def test_segment_tables_that_lie_stay_inside(K):
    """Entries past the rows, or descending, read and write nothing outside."""
    M, N, Kd = 100, 128, 128
    x, xs, w, ws, _ = product_inputs(M, N, Kd, 4, False)
    for bad in ([0, 50, 20, 400, 100], [-5, 10, 2 ** 31 - 1, 30, -2 ** 31], [100, 100, 100, 100, 100]):
        seg = torch.tensor(bad, dtype=I32, device="cuda")
        out, work = K.kmoe_gemm_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), seg)
        no_error(K, work)
        q = [K.kmoe_quantize_fp8_cols(torch.ones(M, c, dtype=BF, device="cuda"), seg) for c in (N, Kd)]
        _, work = K.kmoe_gemm_fp8_wgrad(*q[0], *q[1], seg_start=seg)
        no_error(K, work)


@pytest.mark.parametrize("M,N,Kd,E", [(100, 128, 4096, 512), (300, 256, 4096, 8)])
def test_overlapping_segments_end(K, M, N, Kd, E):
    """More tiles than any ascending table gives, where clusters share items."""
    x, xs = K.kmoe_quantize_fp8(randn(1, M, Kd).to(BF).cuda())
    w, ws = K.kmoe_quantize_fp8_weights(randn(2, 1, N, Kd).to(BF).cuda())
    seg = torch.tensor([0, M] * E, dtype=I32, device="cuda")[:E + 1].contiguous()
    out, work = K.kmoe_gemm_fp8(x, xs, w.repeat(E, 1, 1), ws.repeat(E, 1, 1), seg, out_dtype=F32)
    no_error(K, work)
    # every expert has the same weights, and the first one's tiles come first
    ref, mag = P.gemm(P.values_rows(x.cpu().numpy(), xs.cpu().numpy()),
                      P.values_weights(w.cpu().numpy(), ws.cpu().numpy()), [0, M])
    within(out, ref, product_tolerance(ref, mag, Kd, F32), "out")


def test_weight_gradient_of_many_rows(K):
    rows, N, Kd = 65536, 144, 128
    dy, x = randn(1, rows, N).to(BF).cuda(), randn(2, rows, Kd).to(BF).cuda()
    qd, qx = K.kmoe_quantize_fp8_cols(dy), K.kmoe_quantize_fp8_cols(x)
    dw, work = K.kmoe_gemm_fp8_wgrad(*qd, *qx)
    no_error(K, work)
    ref, mag = P.wgrad(*(P.values_cols(c.cpu().numpy(), s.cpu().numpy()) for c, s in (qd, qx)), [0, rows])
    within(dw, ref, product_tolerance(ref, mag, rows, F32), "dw")


def test_products_past_2_31_elements(K):
    M, N, Kd = 140000, 16384, 128  # M * N > 2^31
    last = M // 64 * 64  # these rows are the first ones again
    x = randn(1, 64, Kd).to(BF).cuda().repeat(-(-M // 64), 1)[:M].contiguous()
    w, ws = K.kmoe_quantize_fp8_weights(randn(2, 1, N, Kd).to(BF).cuda())
    wv = P.values_weights(w.cpu().numpy(), ws.cpu().numpy())
    xc, xs = K.kmoe_quantize_fp8(x)
    out, work = K.kmoe_gemm_fp8(xc, xs, w, ws)
    no_error(K, work)
    assert torch.equal(out[last:last + 16], out[:16])
    ref, mag = P.gemm(P.values_rows(xc[:16].cpu().numpy(), xs[:, :16].cpu().numpy()), wv, [0, 16])
    within(out[:16], ref, product_tolerance(ref, mag, Kd, BF), "out")
    # and back: rows of codes past 2^31
    fc, fs = K.kmoe_quantize_fp8(out[:16].contiguous())
    oc, osc = K.kmoe_quantize_fp8(out)
    del out
    for at in (0, last):
        assert torch.equal(oc[at:at + 16], fc) and torch.equal(osc[:, at:at + 16], fs)
    back, work = K.kmoe_gemm_fp8(oc, osc, w, ws, transpose=True, out_dtype=F32, workspace=work)
    no_error(K, work)
    assert torch.equal(back[last:last + 16], back[:16])
    ref, mag = P.gemm(P.values_rows(fc.cpu().numpy(), fs.cpu().numpy()), wv, [0, 16], transpose=True)
    within(back[:16], ref, product_tolerance(ref, mag, N, F32), "back")


@pytest.mark.parametrize("rows", [900, 30000])
def test_weights_past_2_31_elements(K, rows):
    E, N, Kd = 300, 4096, 2048  # E * N * K > 2^31
    seg = segments(rows, rows, E, behind=0)
    w = torch.randint(0, 0x7F, (E, N, Kd), dtype=U8, device="cuda")  # no NaN codes
    ws = torch.rand(E, N // 128, Kd // 128, device="cuda")
    xc, xs = K.kmoe_quantize_fp8(randn(1, rows, Kd).to(BF).cuda())
    out, work = K.kmoe_gemm_fp8(xc, xs, w, ws, torch.from_numpy(seg).cuda(), out_dtype=F32)
    no_error(K, work)
    for e in np.flatnonzero(np.diff(seg))[[0, -1]]:
        a, b = seg[e], min(seg[e + 1], seg[e] + 4)
        v = P.values_rows(xc[a:b].cpu().numpy(), xs[:, a:b].cpu().numpy())
        ref, mag = P.gemm(v, P.values_weights(w[e:e + 1].cpu().numpy(), ws[e:e + 1].cpu().numpy()), [0, b - a])
        within(out[a:b], ref, product_tolerance(ref, mag, Kd, F32), f"expert {e}")
    del out
    # and their gradient, as large
    dc, ds = K.kmoe_quantize_fp8_cols(randn(2, rows, N).to(BF).cuda(), torch.from_numpy(seg).cuda())
    qc, qs = K.kmoe_quantize_fp8_cols(randn(3, rows, Kd).to(BF).cuda(), torch.from_numpy(seg).cuda())
    dw, work = K.kmoe_gemm_fp8_wgrad(dc, ds, qc, qs, seg_start=torch.from_numpy(seg).cuda())
    no_error(K, work)
    blocks = np.concatenate([[0], np.cumsum(-(-np.diff(seg) // 128))])
    for e in np.flatnonzero(np.diff(seg))[[0, -1]]:
        at, sb = slice(blocks[e] * 128, blocks[e + 1] * 128), slice(blocks[e], blocks[e + 1])
        vd = P.values_cols(dc[at, :256].cpu().numpy(), ds[sb, :256].cpu().numpy())
        vx = P.values_cols(qc[at].cpu().numpy(), qs[sb].cpu().numpy())
        ref, mag = P.wgrad(vd, vx, [0, seg[e + 1] - seg[e]])
        within(dw[e:e + 1, :256], ref, product_tolerance(ref, mag, seg[e + 1] - seg[e] + 128, F32), f"dw {e}")


# ---------------------------------------------------------------- together


def expert_layer(K, x, ids, tw, w, ws, E, d_out):
    """The rows sorted and quantised, one product, the way back, and every gradient."""
    row, slot, seg = K.kmoe_sort_tokens(ids, E)
    xc, xsc = K.kmoe_quantize_fp8(x, row)
    y, work = K.kmoe_gemm_fp8(xc, xsc, w, ws, seg)
    out = K.kmoe_unpermute(y, row, tw)
    d_y, d_w = K.kmoe_unpermute_backward(d_out, y, row, tw)
    gc, gs = K.kmoe_quantize_fp8(d_y)
    d_xp, _ = K.kmoe_gemm_fp8(gc, gs, w, ws, seg, transpose=True, workspace=work)
    d_x = K.kmoe_unpermute(d_xp, row)
    xp = K.kmoe_permute(x, row)
    dw, _ = K.kmoe_gemm_fp8_wgrad(*K.kmoe_quantize_fp8_cols(d_y, seg), *K.kmoe_quantize_fp8_cols(xp, seg),
                                  seg_start=seg, workspace=work)
    return out, d_x, d_w, dw, work


@pytest.mark.parametrize("T,E,k,N,Kd", [(50, 8, 3, 272, 400), (3, 16, 2, 128, 256), (700, 6, 4, 400, 272)])
def test_expert_layer_and_its_gradients(K, T, E, k, N, Kd):
    """The chain against the same chain in 64 bits with the same quantisers: the
    bf16 roundings between the steps (half a unit each) and E4M3's (2^-4 of a
    value, from bf16 inputs that may differ by one rounding and so land on the
    neighbouring code) bound the difference in the 2-norm."""
    ids = routing(T, T, E, k, 0.1)
    x, d_out = randn(1, T, Kd).to(BF), (1e-2 * randn(2, T, N)).to(BF)
    tw = torch.softmax(randn(3, T, k), 1)
    w = (0.05 * randn(4, E, N, Kd)).to(BF)
    wc, ws = K.kmoe_quantize_fp8_weights(w.cuda())
    out, d_x, d_w, dw, work = expert_layer(K, x.cuda(), torch.from_numpy(ids).cuda(), tw.cuda(), wc, ws, E, d_out.cuda())
    no_error(K, work)
    row, slot, seg = P.sort_tokens(ids, E)
    n = int(seg[E])
    token = slot[:n] // k
    wv = P.values_weights(wc.cpu().numpy(), f64(ws))
    xp = f64(x)[token]
    xv = P.values_rows(*P.quantize_rows(xp))
    y = P.gemm(xv, wv, seg)[0]
    ref_out = P.unpermute(y, row, f64(tw))[0]
    d_y, ref_dw, _ = P.unpermute_backward(f64(d_out), np.concatenate([y, np.zeros((T * k - n, N))]), row, f64(tw))
    d_y = f64(torch.from_numpy(d_y[:n]).float().to(BF))
    d_xp = P.gemm(P.values_rows(*P.quantize_rows(d_y)), wv, seg, transpose=True)[0]
    ref_dx = P.unpermute(d_xp, row)[0]
    ref_dW = P.wgrad(P.values_cols(*P.quantize_cols(d_y, seg)), P.values_cols(*P.quantize_cols(xp, seg)), seg)[0]
    for name, got, ref in (("out", out, ref_out), ("d_x", d_x, ref_dx), ("d_w", d_w, ref_dw), ("dw", dw, ref_dW)):
        rel = np.linalg.norm(f64(got) - ref) / max(np.linalg.norm(ref), 1e-30)
        # two bf16 roundings (y or d_xp, then out) and, behind a product of re-rounded rows, codes that differ by a step
        # where the fp32 and the 64-bit product of w and d_out round to bf16 neighbours
        assert rel <= 2 * UBF, (name, rel)


def test_calls_on_a_stream_and_in_a_graph(K):
    T, E, k, N, Kd = 200, 8, 3, 272, 400
    ids = torch.from_numpy(routing(T, T, E, k, 0.1)).cuda()
    x, d_out = randn(1, T, Kd).to(BF).cuda(), (1e-2 * randn(2, T, N)).to(BF).cuda()
    tw = torch.softmax(randn(3, T, k), 1).cuda()
    wc, ws = K.kmoe_quantize_fp8_weights((0.05 * randn(4, E, N, Kd)).to(BF).cuda())
    row, slot, seg = K.kmoe_sort_tokens(ids, E)
    n = int(seg[E])
    first = expert_layer(K, x, ids, tw, wc, ws, E, d_out)[:4]
    again = expert_layer(K, x, ids, tw, wc, ws, E, d_out)[:4]
    for a, b in zip(first, again):
        assert torch.equal(a, b)  # no order of execution changes a bit
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = expert_layer(K, x, ids, tw, wc, ws, E, d_out)[:4]
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(first, other):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = expert_layer(K, x, ids, tw, wc, ws, E, d_out)[:4]
    x2 = randn(9, T, Kd).to(BF).cuda()
    ids2 = torch.from_numpy(routing(T + 1, T, E, k, 0.2)).cuda()
    want = expert_layer(K, x2, ids2, tw, wc, ws, E, d_out)[:4]
    x.copy_(x2)
    ids.copy_(ids2)
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(captured, want):
        assert torch.equal(a, b)


def test_calls_at_once(K):
    """Products, gradients and moves on two streams, each call with its own workspace."""
    x, d = randn(1, 600, 1040).to(BF).cuda(), randn(2, 600, 528).to(BF).cuda()
    wc, ws = K.kmoe_quantize_fp8_weights(randn(3, 1, 528, 1040).to(BF).cuda())
    ids = torch.from_numpy(routing(4, 600, 9, 4, 0.1)).cuda()
    tw = torch.softmax(randn(5, 600, 4), 1).cuda()

    def run():
        xc, xs = K.kmoe_quantize_fp8(x)
        few, w1 = K.kmoe_gemm_fp8(xc[:7].contiguous(), xs[:, :7].contiguous(), wc, ws)
        many, w2 = K.kmoe_gemm_fp8(xc, xs, wc, ws)
        dw, w3 = K.kmoe_gemm_fp8_wgrad(*K.kmoe_quantize_fp8_cols(d), *K.kmoe_quantize_fp8_cols(x))
        row, _, _ = K.kmoe_sort_tokens(ids, 9)
        xp = K.kmoe_permute(x, row, out=torch.zeros(2400, 1040, dtype=BF, device="cuda"))
        return [few, many, dw, row, K.kmoe_unpermute(xp, row, tw)], [w1, w2, w3]

    want, _ = run()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(run())
    torch.cuda.synchronize()
    for outs, works in got:
        for w in works:
            no_error(K, w)
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_rows_that_are_none(K):
    """Entries of row_of_slot outside the rows count as -1 in every call."""
    T, H, E, k = 70, 144, 6, 3
    _, row, _ = sorted_rows(T, E, k, 0.2)
    bad = row.copy()
    none = np.argwhere(row < 0)
    assert len(none) >= 4
    for (t, j), v in zip(none, [T * k, 2 ** 31 - 1, -2 ** 31, -7] * len(none)):
        bad[t, j] = v
    r, b = torch.from_numpy(row).cuda(), torch.from_numpy(bad).cuda()
    x, y, w = randn(1, T, H).to(BF).cuda(), randn(2, T * k, H).to(BF).cuda(), randn(3, T, k).cuda()

    def run(rows):
        out = torch.zeros_like(y)
        d_y = torch.zeros_like(y)
        q = torch.zeros(T * k, H, dtype=U8, device="cuda"), torch.zeros(2, T * k, device="cuda")
        K.kmoe_permute(x, rows, out=out)
        K.kmoe_quantize_fp8(x, rows, codes=q[0], scales=q[1])
        return [out, K.kmoe_unpermute(y, rows, w), *K.kmoe_unpermute_backward(x, y, rows, w, d_y=d_y), *q]

    for got, want in zip(run(b), run(r)):
        assert torch.equal(got, want)


def test_quantize_into_many_sorted_rows_without_a_workspace(K):
    T, cols, E, k = 4100, 144, 40, 16
    x = special(T, T, cols).cuda()
    _, row, seg = sorted_rows(T, E, k)
    r, n = torch.from_numpy(row).cuda(), int(seg[E])
    codes, scales = K.kmoe_quantize_fp8(x, r)
    c2, s2 = torch.empty_like(codes), torch.empty_like(scales)
    st = torch.cuda.current_stream().cuda_stream
    assert K._lib.kmoe_quantize_fp8(x.data_ptr(), T, cols, r.data_ptr(), k, c2.data_ptr(), s2.data_ptr(), None, 0, st) == 0
    assert torch.equal(c2[:n], codes[:n]) and torch.equal(s2[:, :n], scales[:, :n])
