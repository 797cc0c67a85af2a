"""GPU checks of the operators around the experts against the float64
definitions of oracle.operators.

Tolerances.  A value stored in bf16 is off by at most half a unit in the last
place, 2^-8 of it (2^-24 in fp32); U32 = 2^-24 is the unit of one fp32
operation, and a chain of n of them is off by at most n * U32 of the sum of the
absolute terms."""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import formats as F
from oracle import operators as P
from tests._moe_setup import device_inputs, device_weights, params

pytestmark = pytest.mark.gpu
U32, UBF = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def K():
    import mxfp8_mxfp4_moe_gb300 as K
    assert K.kmoe_check_device(0) == 0
    return K


def randn(seed, *shape):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32))


def f64(t):
    return t.detach().double().cpu().numpy()


def at_offset(t, elements):
    """t's values in memory that starts `elements` elements after a 256-byte boundary."""
    buf = torch.empty(t.numel() + elements, dtype=t.dtype, device="cuda")
    v = buf[elements:].view(t.shape)
    v.copy_(t)
    return v


def within(got, ref, tol, what):
    g = f64(got)
    assert g.shape == ref.shape
    bad = ~(np.abs(g - ref) <= tol)  # NaN is off
    i = np.unravel_index(np.argmax(bad), ref.shape) if ref.size else None
    assert not bad.any(), f"{what}: {bad.sum()} of {ref.size} off, at {i}: {g[i]!r} against {ref[i]!r}, {tol[i]!r} allowed"


# ---------------------------------------------------------------- norm

NORM_SHAPES = [(1, 1), (3, 33), (5, 128), (2, 7168), (9, 4104), (4, 5001), (1, 32768), (2, 31999), (700, 64),
               (1500, 96), (17, 3584), (333, 1000), (1, 40), (2100, 32)]


def norm_tolerances(x, r, h, y, H, stream):
    """h: the fp32 sum and its rounding.  y: bf16's half unit, and for the
    factor and the two products fp32 chains of at most H + 8 operations (the sum
    of squares in any order, all terms positive; half of that in the root)."""
    ulp = UBF if stream is BF else U32
    tol_h = (ulp + 2 * U32) * np.abs(h) + U32 * (np.abs(x) + np.abs(r))
    # the addition's rounding in front of the norm moves an element by U32 of its summands
    tol_y = (UBF * 1.01 + (H + 16) * U32) * np.abs(y) + 1e-38
    return tol_h, tol_y


@pytest.mark.parametrize("T,H", NORM_SHAPES)
@pytest.mark.parametrize("stream,weight", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
def test_norm(K, T, H, stream, weight):
    x, r = randn(T + H, T, H).to(BF), (3 * randn(T + H + 1, T, H)).to(stream)
    w = (1 + 0.1 * randn(H, H)).to(weight)
    mx = H % 32 == 0
    h, y, codes, scales = K.kmoe_rmsnorm(x.cuda(), w.cuda(), residual=r.cuda(), eps=1e-5, mx=mx)
    hr, yr = P.rmsnorm(f64(x), f64(r), f64(w), 1e-5)
    tol_h, tol_y = norm_tolerances(f64(x), f64(r), hr, yr, H, stream)
    within(h, hr, tol_h, "h")
    # where x and r cancel, h itself carries the addition's rounding into y
    rstd = 1 / np.sqrt((hr * hr).mean(1, keepdims=True) + 1e-5)
    within(y, yr, tol_y + U32 * (np.abs(f64(x)) + np.abs(f64(r))) * rstd * np.abs(f64(w)) * 2, "y")
    if mx:
        cr, sr = F.quantize_mx(F.bf16_decode(y.cpu().view(torch.int16).numpy()))
        assert np.array_equal(codes.cpu().numpy(), cr) and np.array_equal(scales.cpu().numpy(), sr)


@pytest.mark.parametrize("T,H", [(1, 128), (40, 7168), (1100, 256)])
def test_norm_codes_are_the_quantised_rows(K, T, H):
    x, w = randn(5, T, H).to(BF).cuda(), randn(6, H).cuda()
    _, y, codes, scales = K.kmoe_rmsnorm(x, w, mx=True)
    c, s = K.kmoe_quantize_mx(y)
    assert torch.equal(codes, c) and torch.equal(scales, s)


def test_norm_without_residual_and_in_place(K):
    T, H = 37, 4096
    x, r, w = randn(1, T, H).to(BF).cuda(), randn(2, T, H).to(BF).cuda(), randn(3, H).to(BF).cuda()
    h0, y0, c, s = K.kmoe_rmsnorm(x, w)
    assert h0 is None and c is None and s is None
    _, yr = P.rmsnorm(f64(x), None, f64(w), 1e-6)
    within(y0, yr, (UBF * 1.01 + (H + 16) * U32) * np.abs(yr) + 1e-38, "y")
    h1, y1, _, _ = K.kmoe_rmsnorm(x, w, residual=r)
    keep = r.clone()
    h2, y2, _, _ = K.kmoe_rmsnorm(x, w, residual=keep, h=keep)
    assert h2 is keep and torch.equal(h2, h1) and torch.equal(y2, y1)


@pytest.mark.parametrize("H", [64, 2560, 1003])
@pytest.mark.parametrize("off", [1, 2, 5])
def test_norm_at_any_alignment(K, H, off):
    """Rows that start inside a 16-byte word give the values of aligned ones."""
    T = 21
    x, r, w = randn(1, T, H).to(BF), randn(2, T, H), randn(3, H).to(BF)
    dy, di = randn(4, T, H).to(BF), randn(5, T, H)
    a = K.kmoe_rmsnorm(x.cuda(), w.cuda(), residual=r.cuda())
    b = K.kmoe_rmsnorm(at_offset(x, off), at_offset(w, off), residual=at_offset(r, off), h=at_offset(r, off),
                       y=at_offset(x, off))
    # another split of the row may round the sum of squares otherwise
    _, yr = P.rmsnorm(f64(x), f64(r), f64(w), 1e-6)
    assert torch.equal(a[0], b[0])
    within(b[1], f64(a[1]), 2 * UBF * np.abs(yr) + 1e-38, "y")
    g = K.kmoe_rmsnorm_backward(dy.cuda(), r.cuda(), w.cuda(), dh_in=di.cuda())
    q = K.kmoe_rmsnorm_backward(at_offset(dy, off), at_offset(r, off), at_offset(w, off), dh_in=at_offset(di, off),
                                dh=at_offset(r, off), dweight=at_offset(torch.zeros(H), off))
    ref = P.rmsnorm_backward(f64(dy), f64(r), f64(w), f64(di), 1e-6)
    for got in (g, q):
        check_norm_gradient(got, ref, dy, r, w, di, 1e-6)


def test_norm_codes_at_any_alignment(K):
    T, H = 19, 160
    x, r, w = randn(1, T, H).to(BF), randn(2, T, H), randn(3, H)
    h, y, codes, scales = K.kmoe_rmsnorm(at_offset(x, 1), at_offset(w, 1), residual=at_offset(r, 1), mx=True)
    c, s = K.kmoe_quantize_mx(torch.nn.functional.pad(y, (0, 256 - H)))  # that call wants multiples of 128 columns
    assert torch.equal(codes, c[:, :H]) and torch.equal(scales, s[:, :H // 32])
    ref = K.kmoe_rmsnorm(x.cuda(), w.cuda(), residual=r.cuda(), mx=True)
    assert torch.equal(h, ref[0])


def test_norm_special_rows(K):
    """Zero rows, subnormals, infinities and NaN, each in a row of its own."""
    H = 256
    x = randn(1, 8, H)
    x[0] = 0
    x[1] = 1e-39
    x[2, 5] = float("inf")
    x[3, 7] = float("nan")
    x[4, 1:] = 0
    x[5] *= 1e15
    x[6] *= 1e-15
    x, w = x.to(BF), (1 + 0.1 * randn(2, H)).to(BF)
    r = torch.zeros(8, H)
    h, y, codes, scales = K.kmoe_rmsnorm(x.cuda(), w.cuda(), residual=r.cuda(), eps=1e-6, mx=True)
    with np.errstate(invalid="ignore"):
        _, yr = P.rmsnorm(f64(x), f64(r), f64(w), 1e-6)
    assert torch.equal(h.cpu().isnan(), x.isnan()) and torch.equal(h.cpu()[~x.isnan()], x.float()[~x.isnan()])
    assert np.array_equal(np.isnan(f64(y)), np.isnan(yr))
    ok = ~np.isnan(yr)
    assert np.all(np.abs(f64(y) - yr)[ok] <= (UBF * 1.01 + (H + 16) * U32) * np.abs(yr[ok]) + 2.0 ** -133)
    c, s = K.kmoe_quantize_mx(y)
    assert torch.equal(codes, c) and torch.equal(scales, s)
    assert scales.max() < 255


def check_norm_gradient(got, ref, dy, h, w, d_in, eps):
    """dh: its storage's half unit, and fp32 chains (at most H + 32
    operations) over the terms' absolute values.  dweight: chains of at most
    T + 16 over rows whose factor is off by H + 8 units."""
    dh, dw = got
    T, H = ref[0].shape
    dyn, hn, wn = f64(dy), f64(h), f64(w)
    rstd = 1 / np.sqrt((hn * hn).mean(1, keepdims=True) + eps)
    n, g = hn * rstd, dyn * wn
    size = rstd * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(1, keepdims=True))
    if d_in is not None:
        size = size + np.abs(f64(d_in))
    ulp = UBF if dh.dtype is BF else U32
    within(dh, ref[0], ulp * 1.01 * np.abs(ref[0]) + (H + 32) * U32 * size + 1e-38, "dh")
    within(dw, ref[1], (T + H + 32) * U32 * np.abs(dyn * n).sum(0) + 1e-38, "dweight")


@pytest.mark.parametrize("T,H", NORM_SHAPES)
@pytest.mark.parametrize("stream,weight", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
def test_norm_gradient(K, T, H, stream, weight):
    dy, h = (1e-2 * randn(T + H, T, H)).to(BF), (3 * randn(T + H + 1, T, H)).to(stream)
    w, d_in = (1 + 0.1 * randn(H, H)).to(weight), (1e-2 * randn(T + H + 2, T, H)).to(stream)
    got = K.kmoe_rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), dh_in=d_in.cuda(), eps=1e-5)
    check_norm_gradient(got, P.rmsnorm_backward(f64(dy), f64(h), f64(w), f64(d_in), 1e-5), dy, h, w, d_in, 1e-5)
    got = K.kmoe_rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), eps=1e-5)
    check_norm_gradient(got, P.rmsnorm_backward(f64(dy), f64(h), f64(w), None, 1e-5), dy, h, w, None, 1e-5)


def test_norm_gradient_in_place_empty_and_repeated(K):
    T, H = 1234, 640
    dy, h, w = randn(1, T, H).to(BF).cuda(), randn(2, T, H).to(BF).cuda(), randn(3, H).cuda()
    d_in = randn(4, T, H).to(BF).cuda()
    dh, dw = K.kmoe_rmsnorm_backward(dy, h, w, dh_in=d_in)
    keep = d_in.clone()
    ws = torch.full((K.kmoe_rmsnorm_workspace_size(T, H),), 255, dtype=torch.uint8, device="cuda")  # NaN words
    dh2, dw2 = K.kmoe_rmsnorm_backward(dy, h, w, dh_in=keep, dh=keep, workspace=ws)
    assert dh2 is keep and torch.equal(dh, dh2) and torch.equal(dw, dw2)  # fixed summation order
    e = torch.empty(0, H, dtype=BF, device="cuda")
    dw0 = torch.full((H,), 7.0, device="cuda")
    K.kmoe_rmsnorm_backward(e, e, w, dweight=dw0)
    assert torch.all(dw0 == 0)
    assert K.kmoe_rmsnorm(e, w)[1].shape == (0, H)


def test_norm_rows_past_31_bits(K):
    """Element offsets beyond 2^31: the last rows of a tall batch."""
    H = 8192
    T = (1 << 31) // H + 5
    x = torch.zeros(T, H, dtype=BF, device="cuda")
    tail = randn(1, 5, H).to(BF).cuda()
    x[-5:] = tail
    w = randn(2, H).cuda()
    y = K.kmoe_rmsnorm(x, w)[1]
    assert torch.equal(y[-5:], K.kmoe_rmsnorm(tail, w)[1]) and not y[:1000].any()
    dy = torch.zeros_like(x)
    dy[-5:] = tail.flip(0)
    dh, dw = K.kmoe_rmsnorm_backward(dy, x, w, dh=y)
    assert torch.equal(dh[-5:], K.kmoe_rmsnorm_backward(tail.flip(0).contiguous(), tail, w)[0])


# ---------------------------------------------------------------- routing

ROUTE_SHAPES = [  # T, E, k, n_group, topk_group
    (33, 896, 16, 8, 4), (16, 896, 16, 1, 1), (50, 256, 8, 8, 4), (7, 1024, 32, 32, 17), (40, 64, 6, 1, 1),
    (3, 1, 1, 1, 1), (9, 5, 5, 1, 1), (21, 37, 5, 1, 1), (12, 160, 6, 8, 3), (10, 32, 8, 32, 9), (5, 1000, 31, 4, 1),
    (1, 896, 1, 2, 1), (300, 128, 8, 1, 1), (6, 1024, 32, 1, 1), (11, 96, 32, 3, 2), (8, 40, 20, 20, 10)]


def check_route(K, logits, bias, k, n_group, topk_group, softmax, renormalize, scale):
    ids, w = K.kmoe_route_grouped(logits.cuda(), None if bias is None else bias.cuda(), k,
                                  score="softmax" if softmax else "sigmoid", n_group=n_group, topk_group=topk_group,
                                  renormalize=renormalize, scale=scale)
    ri, rw = P.route_grouped(logits.numpy(), None if bias is None else bias.numpy(), k, softmax, n_group, topk_group,
                             renormalize, scale)
    assert np.array_equal(ids.cpu().numpy(), ri)
    # a score is at most 16 fp32 operations, and its exponential's argument at most as far off as the logits are large
    l = logits.double().numpy()
    size = np.where(np.isfinite(l), np.abs(l), 0.0).max(1, keepdims=True)
    within(w, rw, (40 + 4 * size + (logits.shape[1] if softmax else k)) * U32 * np.abs(rw) + 1e-37, "weights")
    return ids, w


@pytest.mark.parametrize("T,E,k,G,Kg", ROUTE_SHAPES)
@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("renormalize,scale", [(True, 2.5), (False, 1.0)])
def test_route_grouped(K, T, E, k, G, Kg, softmax, with_bias, renormalize, scale):
    logits = 1.7 * randn(T + E, T, E)
    bias = 0.1 * randn(E, E) if with_bias else None
    check_route(K, logits, bias, k, G, Kg, softmax, renormalize, scale)


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_ties(K, softmax, with_bias):
    """Logits and biases of few values: equal keys in every row, equal groups."""
    T, E = 64, 256
    logits = torch.round(2 * randn(1, T, E)) / 2
    logits[0] = 0
    logits[1] = torch.arange(E) % 2
    logits[2] = 30.0 + torch.arange(E) % 3      # sigmoids that are all 1
    logits[3] = -30.0 - torch.arange(E) % 3
    bias = torch.round(4 * randn(2, E)) / 32 if with_bias else None
    for k, G, Kg in ((8, 8, 4), (32, 1, 1), (16, 16, 3), (1, 32, 1)):
        check_route(K, logits, bias, k, G, Kg, softmax, True, 1.0)
    if with_bias:
        check_route(K, logits, torch.zeros(E), 8, 8, 4, softmax, True, 1.0)


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_near_ties(K, softmax, with_bias):
    """Keys a few units in the last place apart: only the exact scores order them."""
    T, E = 64, 224
    step = torch.from_numpy(np.random.default_rng(7).integers(-6, 7, (T, E)).astype(np.float32))
    logits = (1.0 + step * 2.0 ** -23)
    bias = 0.25 + torch.from_numpy(np.random.default_rng(8).integers(0, 3, E).astype(np.float32)) * 2.0 ** -24 \
        if with_bias else None
    for k, G, Kg in ((8, 1, 1), (32, 1, 1), (16, 7, 2)):
        check_route(K, logits, bias, k, G, Kg, softmax, True, 1.0)
    # a few near-equal keys at the cut among well separated ones
    logits = 1.7 * randn(3, T, E)
    top = logits.topk(12, dim=1).values[:, 7:8]
    logits = torch.where((logits - top).abs() < 0.3, top + step[:, :E] * 2.0 ** -22, logits)
    for k, G, Kg in ((8, 1, 1), (9, 7, 5)):
        check_route(K, logits, None if bias is None else torch.full((E,), 0.5), k, G, Kg, softmax, True, 1.0)


@pytest.mark.parametrize("softmax", [False, True])
def test_route_near_tie_behind_equal_keys(K, softmax):
    """Many equal keys at the cut, and behind them by index one that exceeds
    them by less than a cheap key tells."""
    T, E = 40, 64
    logits = torch.full((T, E), -1.0)
    for t in range(T):
        logits[t, (7 * t) % E] += 2.0 ** -23 * (1 + t % 3)
    logits[:, :2] = 2.0
    for bias in (torch.zeros(E), torch.full((E,), 0.25)):
        for k, G, Kg in ((6, 1, 1), (20, 1, 1), (31, 8, 5)):
            check_route(K, logits, bias, k, G, Kg, softmax, True, 1.0)
    low = torch.full((T, E), torch.finfo(torch.float32).min)
    low[:, 0] = 1.0
    low[torch.arange(T), 5 + torch.arange(T) % 50] = -80.0
    check_route(K, low, torch.zeros(E), 4, 1, 1, softmax, False, 1.0)
    check_route(K, low, torch.zeros(E), 4, 8, 2, softmax, False, 1.0)


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_masked_and_non_finite(K, softmax, with_bias, renormalize):
    """Rows with masked experts, with fewer experts than slots, with none; NaN and infinite logits and biases."""
    T, E, k, G, Kg = 12, 64, 6, 8, 3
    logits = 1.7 * randn(1, T, E)
    logits[0] = -float("inf")
    logits[1, 5:] = -float("inf")
    logits[2, :60] = -float("inf")
    logits[3, ::8] = float("nan")
    logits[4] = float("nan")
    logits[5, 3] = float("inf")
    logits[6, 1::2] = -float("inf")
    logits[7, :] = -float("inf")
    logits[7, ::8] = 1.0                          # one expert a group
    logits[8] = -3.0e38                           # the type's lowest values
    logits[9] *= 50
    logits[10, 9:11] = float("inf")
    logits[11, 1:] = torch.finfo(torch.float32).min
    bias = None
    if with_bias:
        bias = 0.1 * randn(2, E)
        bias[11], bias[12], bias[13] = float("nan"), -float("inf"), -3.0
    for g, kg in ((1, 1), (G, Kg)):
        check_route(K, logits, bias, k, g, kg, softmax, renormalize, 2.5)


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_masked_with_the_lowest_value(K, softmax, renormalize):
    """Experts masked with finite lows that their bias puts first: they weigh
    nothing, alone or beside others, and have no gradient."""
    T, E, k = 6, 48, 4
    low = torch.finfo(torch.float32).min
    logits, bias = 1.7 * randn(1, T, E), 0.1 * randn(2, E)
    bias[[3, 17, 30, 41]] = 5.0
    logits[0, [3, 17, 30, 41]] = low
    logits[1, [3, 17]] = low
    logits[2] = low
    logits[3, [3, 17, 30, 41]] = torch.tensor([-690.0, -750.0, -699.0, -1e30])
    logits[4, [3, 17, 30, 41]] = -1e4
    ids, w = check_route(K, logits, bias, k, 1, 1, softmax, renormalize, 2.5)
    assert (ids[0].sort().values.cpu() == torch.tensor([3, 17, 30, 41])).all() and not w[0].any()
    d_w = randn(3, T, k)
    got = K.kmoe_route_backward(d_w.cuda(), logits.cuda(), ids, score="softmax" if softmax else "sigmoid",
                                renormalize=renormalize, scale=2.5)
    n = ids.cpu().numpy()
    ref = P.route_backward(d_w.double().numpy(), logits.numpy(), n, softmax, renormalize, 2.5)
    check_route_gradient(got, ref, d_w.double().numpy(), logits, n, softmax, renormalize, 2.5)
    assert not got[0, n[0]].any()


def test_route_matches_the_layers_routing(K):
    w = W.WORKLOADS["decode"]
    inp, _ = device_inputs(w)
    a, aw = K.kmoe_route(inp["logits"], inp["bias"], w.k)
    b, bw = K.kmoe_route_grouped(inp["logits"], inp["bias"], w.k)
    assert torch.equal(a, b)
    assert torch.all((aw - bw).abs() <= 40 * U32 * aw)


def test_route_extreme_logits(K):
    """Scores that underflow, and saturated ones, with weights that still sum to one or are 0."""
    logits = torch.tensor([[-120.0, -200.0, -90.0, -104.0], [88.0, 90.0, 120.0, 3e38], [-3e38, -1e30, -1e20, -1e10]])
    for softmax in (False, True):
        check_route(K, logits, None, 3, 1, 1, softmax, softmax, 1.0)
        check_route(K, logits, torch.zeros(4), 3, 1, 1, softmax, softmax, 1.0)


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("renormalize,scale", [(True, 2.5), (False, 1.0)])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (33, 896, 16), (40, 64, 6), (9, 5, 5), (6, 1024, 32), (500, 160, 6),
                                   (21, 37, 32), (3, 1001, 7), (1, 130, 1)])
def test_route_gradient(K, T, E, k, softmax, renormalize, scale):
    logits, d_w = 1.7 * randn(T + E, T, E), randn(k, T, k)
    ids = P.route_grouped(logits.numpy(), None, k)[0]
    if T > 4:
        ids[3] = -1                     # a row with no expert
        ids[4, k // 2:] = -1
        ids[2, 0] = E                   # outside: masked
        d_w[3] = float("nan")           # not read
    got = K.kmoe_route_backward(d_w.cuda(), logits.cuda(), torch.from_numpy(ids).cuda(),
                                score="softmax" if softmax else "sigmoid", renormalize=renormalize, scale=scale,
                                d_logits=torch.full((T, E), float("nan"), device="cuda"))
    d = np.where((ids >= 0) & (ids < E), d_w.double().numpy(), 0.0)
    ref = P.route_backward(d, logits.numpy(), ids, softmax, renormalize, scale)
    check_route_gradient(got, ref, d, logits, ids, softmax, renormalize, scale)


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient_against_differences(K, softmax, renormalize):
    """The gradient along a direction against differences of the routing's own
    weights.  A step of 2^-7 either way: the weights' roundings (40 units each)
    over it, and the third derivative's share, at most 10 of the weight."""
    T, E, k, step = 200, 96, 6, 2.0 ** -7
    logits, d_w = (1.7 * randn(1, T, E)).cuda(), randn(2, T, k).cuda()
    kw = dict(score="softmax" if softmax else "sigmoid", renormalize=renormalize, scale=2.5)
    ids, w = K.kmoe_route_grouped(logits, None, k, **kw)
    along = torch.where(torch.rand(T, E, generator=torch.Generator().manual_seed(3)) < 0.5, -1.0, 1.0).cuda()
    hi, lo = (K.kmoe_route_grouped(logits + s * along, None, k, **kw) for s in (step, -step))
    same = (hi[0] == ids).all(1) & (lo[0] == ids).all(1)
    assert same.sum() > T // 4
    num = ((hi[1] - lo[1]).double() * d_w.double()).sum(1) / (2 * step)
    got = (K.kmoe_route_backward(d_w, logits, ids, **kw).double() * along.double()).sum(1)
    bound = (40 * U32 / step + 10 * step ** 2) * (d_w.double() * w.double()).abs().sum(1)
    assert torch.all(((num - got).abs() <= bound)[same])


def check_route_gradient(got, ref, d, logits, ids, softmax, renormalize, scale):
    """An element is its score (or share) times a difference of two terms:
    fp32 chains of k + 40 operations over their absolute values (E more in the
    softmax), and the exponential's argument."""
    E = logits.shape[1]
    w = np.abs(P.route_weights(logits.numpy(), ids, softmax, renormalize, scale))
    s = P.scores(logits.numpy(), softmax)
    ok = (ids >= 0) & (ids < E)
    term = np.zeros(ref.shape)
    for j in range(ids.shape[1]):
        term[np.arange(len(ids)), np.where(ok[:, j], ids[:, j], 0)] += np.where(
            ok[:, j], w[:, j] * (np.abs(d[:, j]) + (np.abs(d) * w).sum(1) / scale * (renormalize or softmax)), 0.0)
    if softmax and not renormalize:
        term += s * (np.abs(d) * w).sum(1, keepdims=True)
    l = logits.double().numpy()
    size = np.where(np.isfinite(l), np.abs(l), 0.0).max(1, keepdims=True)
    within(got, ref, (60 + ids.shape[1] + 8 * size + E * softmax) * U32 * term + 1e-37, "d_logits")


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient_special_rows(K, softmax, renormalize):
    """Saturated and masked logits, an expert in two slots."""
    T, E, k = 7, 40, 4
    logits, d_w = 1.7 * randn(1, T, E), randn(2, T, k)
    logits[0] = -float("inf")
    logits[1, 10:] = -float("inf")
    logits[2, 3] = 60.0
    logits[3] = -60.0
    logits[4, 20:] = float("nan")
    ids = np.tile(np.array([3, 0, 7, 5], np.int32), (T, 1))
    ids[5] = [6, 6, 2, 6]
    ids[6] = [-1, 39, -1, 39]
    got = K.kmoe_route_backward(d_w.cuda(), logits.cuda(), torch.from_numpy(ids).cuda(),
                                score="softmax" if softmax else "sigmoid", renormalize=renormalize, scale=2.5)
    d = np.where(ids >= 0, d_w.double().numpy(), 0.0)
    ref = P.route_backward(d, logits.numpy(), ids, softmax, renormalize, 2.5)
    # an expert's slots are added: their absolute terms bound the sum
    check_route_gradient(got, ref, d, logits, ids, softmax, renormalize, 2.5)


# ---------------------------------------------------------------- combine

@pytest.mark.parametrize("T,H,k", [(1, 4, 1), (3, 36, 5), (16, 7168, 16), (129, 3584, 8), (40, 100, 32), (5, 8188, 3),
                                   (200, 128, 16), (2, 32768, 7)])
@pytest.mark.parametrize("masked", [False, True])
def test_combine_gradient(K, T, H, k, masked):
    E = 64
    rng = np.random.default_rng(T + H)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    y, g = randn(T, T * k, H), randn(H, T, H).to(BF)
    if masked:
        ids[rng.random((T, k)) < 0.3] = -1
        ids[0, 0] = E
        if T > 2:
            ids[2] = -1
        y[torch.from_numpy(((ids < 0) | (ids >= E)).reshape(-1))] = float("nan")  # rows the forward never wrote
    got = K.kmoe_combine_backward(g.cuda(), y.cuda(), torch.from_numpy(ids).cuda(), E, 2.5)
    yn = np.nan_to_num(f64(y), nan=0.0).reshape(T, k, H)
    ref = P.combine_backward(f64(g), f64(y), ids, E, 2.5)
    # a chain of at most H products over their absolute values
    within(got, ref, (H + 8) * U32 * 2.5 * np.einsum("tkh,th->tk", np.abs(yn), np.abs(f64(g))) + 1e-37, "d_w")


def test_combine_gradient_rows_past_31_bits(K):
    H, k = 8192, 32
    T = (1 << 31) // (H * k) + 2
    y = torch.zeros(T * k, H, device="cuda")
    g = torch.zeros(T, H, dtype=BF, device="cuda")
    y[-k:], g[-1] = randn(1, k, H).cuda(), randn(2, H).to(BF).cuda()
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    got = K.kmoe_combine_backward(g, y, ids, 64)
    ref = P.combine_backward(f64(g[-1:]), f64(y[-k:]), np.zeros((1, k), np.int32), 64)
    within(got[-1:], ref, (H + 8) * U32 * (y[-k:].double() @ g[-1].double().abs()).abs().cpu().numpy()[None] * 0
           + (H + 8) * U32 * (y[-k:].double().abs() @ g[-1].double().abs()).cpu().numpy()[None], "d_w")
    assert not got[:-1].any()


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("w", [W.WORKLOADS["tiny"], W.Workload("mid", T=300, H=256, I=128, E=16, k=4),
                               W.Workload("one", T=1, H=384, I=128, E=8, k=8)], ids=lambda w: w.name)
def test_forward_on_quantised_rows_equals_forward(K, w):
    wt = device_weights(w)
    inp, _ = device_inputs(w)
    p = params(w)
    ids, tw = K.kmoe_route_grouped(inp["logits"], inp["bias"], w.k, n_group=4, topk_group=4)
    if w.T > 2:
        ids[1, 0] = -1
        ids[2] = -1
    ref, _ = K.kmoe_forward(p, inp["x"], None, None, wt["w13_k"], wt["w2_k"], topk_ids=ids, topk_w=tw)
    codes, scales = K.kmoe_quantize_mx(inp["x"])
    got, ws = K.kmoe_forward_mx(p, codes, scales, ids, tw, wt["w13_k"], wt["w2_k"])
    assert K.kmoe_device_error(ws)[0] == 0
    assert torch.equal(got, ref)


def test_block_from_stream_to_gradients(K):
    """The operators as a block uses them: norm, gate, grouped routing, experts
    on the norm's codes, then the gradients back to the logits and the stream;
    the routing weights' gradient is that of the layer's output."""
    w = W.Workload("block", T=70, H=256, I=128, E=16, k=4)
    wt = device_weights(w)
    x, r = randn(1, w.T, w.H).to(BF).cuda(), (2 * randn(2, w.T, w.H)).to(BF).cuda()
    nw, gate, bias = (1 + 0.1 * randn(3, w.H)).cuda(), 0.1 * randn(4, w.E, w.H), (0.05 * randn(5, w.E)).cuda()
    p = params(w)
    h, y, codes, scales = K.kmoe_rmsnorm(x, nw, residual=r, mx=True)
    logits = y.float() @ gate.cuda().t()
    ids, tw = K.kmoe_route_grouped(logits, bias, w.k, n_group=4, topk_group=2, scale=1.5)
    out, ws = K.kmoe_forward_mx(p, codes, scales, ids, tw, wt["w13_k"], wt["w2_k"])
    assert K.kmoe_device_error(ws)[0] == 0
    stage = K.stage_views(p, ws)["y"]
    d_out = randn(6, w.T, w.H).to(BF).cuda()
    d_w = K.kmoe_combine_backward(d_out, stage, ids, w.E)
    # out is linear in the weights: sum over slots of d_w * w is <d_out, out>, up to out's bf16 rounding
    lhs, rhs = (d_w.double() * tw.double()).sum(1), (d_out.double() * out.double()).sum(1)
    bound = 1.01 * UBF * (d_out.double() * out.double()).abs().sum(1) + 1e-4 * (d_w.double() * tw.double()).abs().sum(1)
    assert torch.all((lhs - rhs).abs() <= bound)
    d_logits = K.kmoe_route_backward(d_w, logits, ids, scale=1.5)
    ref = P.route_backward(f64(d_w), logits.cpu().numpy(), ids.cpu().numpy(), False, True, 1.5)
    check_route_gradient(d_logits, ref, f64(d_w), logits.cpu(), ids.cpu().numpy(), False, True, 1.5)
    dy = (d_logits @ gate.cuda()).to(BF)
    dh, dnw = K.kmoe_rmsnorm_backward(dy, h, nw, dh_in=d_out)
    check_norm_gradient((dh, dnw), P.rmsnorm_backward(f64(dy), f64(h), f64(nw), f64(d_out), 1e-6), dy, h, nw, d_out,
                        1e-6)


def test_example_learns(K):
    """The example's block runs and its gate learns from the gradients."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses = mod.main(steps=20)
    assert all(np.isfinite(losses)) and losses[-1] < losses[0]


def test_norm_codes_of_infinite_and_huge_values(K):
    """A bf16 row with infinities quantises as kmoe_quantize_mx has it: the
    scale byte 254, finite neighbours scaled by 2^-127."""
    H = 128
    x = randn(1, 4, H).to(BF).cuda()
    w = torch.ones(H)
    w[3], w[4], w[40], w[41] = float("inf"), 3e38, 3e38, -2e38
    _, y, codes, scales = K.kmoe_rmsnorm(x, w.cuda(), mx=True)
    c, s = K.kmoe_quantize_mx(y)
    assert torch.equal(codes, c) and torch.equal(scales, s) and (scales == 254).any()
    cr, sr = F.quantize_mx(F.bf16_decode(y.cpu().view(torch.int16).numpy()))
    assert np.array_equal(codes.cpu().numpy(), cr) and np.array_equal(scales.cpu().numpy(), sr)


def test_route_unaligned_rows(K):
    """Logits and bias that start inside a 16-byte word, and odd expert counts, take the scalar loads."""
    T, E, k = 37, 96, 8
    logits, bias = 1.7 * randn(1, T, E), 0.1 * randn(2, E)
    ri, rw = P.route_grouped(logits.numpy(), bias.numpy(), k, False, 8, 4)
    for o1, o2 in ((1, 0), (0, 2), (3, 5)):
        ids, w = K.kmoe_route_grouped(at_offset(logits, o1), at_offset(bias, o2), k, n_group=8, topk_group=4)
        assert np.array_equal(ids.cpu().numpy(), ri)
    d_w = randn(3, T, k)
    ref = K.kmoe_route_backward(d_w.cuda(), logits.cuda(), ids, score="softmax", renormalize=False)
    got = K.kmoe_route_backward(d_w.cuda(), at_offset(logits, 1), ids, score="softmax", renormalize=False,
                                d_logits=at_offset(torch.zeros(T, E), 3))
    check_route_gradient(got, P.route_backward(d_w.double().numpy(), logits.numpy(), ri, True, False, 1.0),
                         d_w.double().numpy(), logits, ri, True, False, 1.0)
    assert torch.allclose(got, ref, rtol=1e-5, atol=1e-7)


def test_streams_and_graphs(K):
    """On a stream of its own, outputs allocated by the calls; then captured
    once and replayed on new inputs."""
    T, H, E, k = 65, 512, 64, 6
    x, r, w = randn(1, T, H).to(BF).cuda(), randn(2, T, H).to(BF).cuda(), randn(3, H).cuda()
    lg, d_w = randn(4, T, E).cuda(), randn(5, T, k).cuda()
    y3 = randn(6, T * k, H).cuda()
    bias = (0.1 * randn(7, E)).cuda()

    def calls(stream=None):
        h, y, c, s = K.kmoe_rmsnorm(x, w, residual=r, mx=True, stream=stream)
        ids, tw = K.kmoe_route_grouped(lg, bias, k, n_group=8, topk_group=4, stream=stream)
        return [h, y, c, s, ids, tw, K.kmoe_route_backward(d_w, lg, ids, stream=stream),
                K.kmoe_combine_backward(x, y3, ids, E, stream=stream),
                *K.kmoe_rmsnorm_backward(y, h, w, dh_in=x, stream=stream)]
    ref = calls()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = calls(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = calls()
    x.copy_(randn(11, T, H).to(BF))
    lg.copy_(randn(14, T, E))
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(calls(), cap))
