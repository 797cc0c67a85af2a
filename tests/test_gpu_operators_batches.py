"""The operators around the experts at batches that give every row team several
rows: ring slots used again, several rows a team in the weight gradient, block
counts rounded for ragged rows, one warp a token for many tokens.  Random data
in every row, against the float64 definitions; tolerances as in
test_gpu_operators."""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import formats as F
from oracle import operators as P
from tests._moe_setup import device_inputs, device_weights, params
from tests.test_gpu_operators import (BF, F32, K, U32, at_offset, check_norm_gradient, check_route,  # noqa: F401
                                      check_route_gradient, f64, norm_tolerances, randn, within)

pytestmark = pytest.mark.gpu

# warps and blocks a row; one, two and four chunks a thread; even and ragged; past the registers' width
SHAPES = [(11000, 64), (6000, 33), (5000, 416), (5200, 1000), (5100, 1003), (1300, 2056), (700, 3585), (700, 5001),
          (620, 7168), (500, 9001), (400, 16384), (330, 16390)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("stream", [BF, F32])
@pytest.mark.parametrize("with_residual", [True, False])
def test_norm_over_many_rows(K, T, H, stream, with_residual):  # noqa: F811
    x, w = randn(T + H, T, H).to(BF), 1 + 0.1 * randn(H, H)
    r = (3 * randn(T + H + 1, T, H)).to(stream) if with_residual else None
    mx = H % 32 == 0
    on = None if r is None else r.cuda()
    h, y, codes, scales = K.kmoe_rmsnorm(x.cuda(), w.cuda(), residual=on, eps=1e-5, mx=mx)
    rn = None if r is None else f64(r)
    hr, yr = P.rmsnorm(f64(x), rn, f64(w), 1e-5)
    size = np.abs(f64(x)) + (0.0 if r is None else np.abs(rn))
    tol_h, tol_y = norm_tolerances(f64(x), 0.0 * f64(x) if r is None else rn, hr, yr, H, stream)
    rstd = 1 / np.sqrt((hr * hr).mean(1, keepdims=True) + 1e-5)
    within(y, yr, tol_y + 2 * U32 * size * rstd * np.abs(f64(w)), "y")
    if mx:
        c, s = F.quantize_mx(F.bf16_decode(y.cpu().view(torch.int16).numpy()))
        assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)
    if r is not None:
        within(h, hr, tol_h, "h")
        h2, y2, c2, s2 = K.kmoe_rmsnorm(x.cuda(), w.cuda(), residual=on, h=on, eps=1e-5, mx=mx)
        assert h2 is on and torch.equal(h2, h) and torch.equal(y2, y)
        assert not mx or (torch.equal(c2, codes) and torch.equal(s2, scales))


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("stream", [BF, F32])
def test_norm_gradient_over_many_rows(K, T, H, stream):  # noqa: F811
    dy, h = (1e-2 * randn(T + H, T, H)).to(BF), (3 * randn(T + H + 1, T, H)).to(stream)
    w, d_in = 1 + 0.1 * randn(H, H), (1e-2 * randn(T + H + 2, T, H)).to(stream)
    on = d_in.cuda()
    a = K.kmoe_rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), dh_in=on, eps=1e-5)
    check_norm_gradient(a, P.rmsnorm_backward(f64(dy), f64(h), f64(w), f64(d_in), 1e-5), dy, h, w, d_in, 1e-5)
    b = K.kmoe_rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), dh_in=on, dh=on, eps=1e-5)
    assert b[0] is on and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c = K.kmoe_rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), eps=1e-5)
    check_norm_gradient(c, P.rmsnorm_backward(f64(dy), f64(h), f64(w), None, 1e-5), dy, h, w, None, 1e-5)


@pytest.mark.parametrize("stream", [BF, F32])
def test_norm_and_gradient_unaligned_over_many_rows(K, stream):  # noqa: F811
    """More rows than the element-wise gradient has blocks."""
    T, H = 700, 520
    x, r, w = randn(1, T, H).to(BF), (3 * randn(2, T, H)).to(stream), 1 + 0.1 * randn(3, H)
    h, y, _, _ = K.kmoe_rmsnorm(at_offset(x, 1), w.cuda(), residual=at_offset(r, 1), eps=1e-5)
    hr, yr = P.rmsnorm(f64(x), f64(r), f64(w), 1e-5)
    tol_h, tol_y = norm_tolerances(f64(x), f64(r), hr, yr, H, stream)
    rstd = 1 / np.sqrt((hr * hr).mean(1, keepdims=True) + 1e-5)
    within(h, hr, tol_h, "h")
    within(y, yr, tol_y + 2 * U32 * (np.abs(f64(x)) + np.abs(f64(r))) * rstd * np.abs(f64(w)), "y")
    dy = (1e-2 * randn(4, T, H)).to(BF)
    got = K.kmoe_rmsnorm_backward(at_offset(dy, 1), at_offset(r, 1), w.cuda(), dh_in=at_offset(r, 1), eps=1e-5)
    check_norm_gradient(got, P.rmsnorm_backward(f64(dy), f64(r), f64(w), f64(r), 1e-5), dy, r, w, r, 1e-5)


def test_norm_with_residual_past_31_bits(K):  # noqa: F811
    """All tensors of the norm and its gradient beyond 2^31 elements, the weight's gradient among them."""
    H, n = 8192, 5
    T = (1 << 31) // H + n
    x = torch.zeros(T, H, dtype=BF, device="cuda")
    r, dy = torch.zeros_like(x), torch.zeros_like(x)
    x[-n:], r[-n:], dy[-n:] = (randn(i, n, H).to(BF).cuda() for i in (1, 2, 3))
    w = (1 + 0.1 * randn(4, H)).cuda()
    h, y, codes, scales = K.kmoe_rmsnorm(x, w, residual=r, mx=True)
    short = K.kmoe_rmsnorm(x[-n:], w, residual=r[-n:], mx=True)
    for tall, ref in zip((h, y, codes, scales), short):
        assert torch.equal(tall[-n:], ref) and not tall[:-n].any()
    del codes, scales, x, r
    dh, dw = K.kmoe_rmsnorm_backward(dy, h, w, dh_in=y, dh=y)
    tail = f64(dy[-n:]), f64(h[-n:]), f64(w), f64(short[1])
    ref = P.rmsnorm_backward(*tail, 1e-6)
    check_norm_gradient((dh[-n:], dw), ref, dy[-n:], h[-n:], w, short[1], 1e-6)
    assert not dh[:-n].any()


@pytest.mark.parametrize("T,E,k,G,Kg", [(1300, 896, 16, 8, 4), (1300, 1024, 32, 1, 1), (1250, 1000, 8, 8, 3),
                                        (1300, 513, 20, 3, 2), (1300, 768, 31, 32, 20)])
@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_over_many_tokens(K, T, E, k, G, Kg, softmax, with_bias):  # noqa: F811
    logits = 1.7 * randn(T + E, T, E)
    bias = 0.1 * randn(E, E) if with_bias else None
    logits[5::50, ::3] = -float("inf")
    logits[6::50] = -float("inf")
    logits[7::50, 9] = float("nan")
    logits[8::50] = torch.round(logits[8::50])
    check_route(K, logits, bias, k, G, Kg, softmax, True, 2.5)


@pytest.mark.parametrize("T,E,k", [(700, 896, 16), (650, 1024, 32), (1000, 130, 6), (700, 601, 8)])
@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("renormalize,scale", [(True, 2.5), (False, 1.0)])
def test_route_gradient_over_many_tokens(K, T, E, k, softmax, renormalize, scale):  # noqa: F811
    logits, d_w = 1.7 * randn(T + E, T, E), randn(k, T, k)
    ids = P.route_grouped(logits.numpy(), None, k)[0]
    ids[3::40] = -1
    ids[4::40, k // 2:] = -1
    ids[2::40, 0] = E
    got = K.kmoe_route_backward(d_w.cuda(), logits.cuda(), torch.from_numpy(ids).cuda(),
                                score="softmax" if softmax else "sigmoid", renormalize=renormalize, scale=scale,
                                d_logits=torch.full((T, E), float("nan"), device="cuda"))
    d = np.where((ids >= 0) & (ids < E), d_w.double().numpy(), 0.0)
    check_route_gradient(got, P.route_backward(d, logits.numpy(), ids, softmax, renormalize, scale), d, logits, ids,
                         softmax, renormalize, scale)


@pytest.mark.parametrize("w", [W.Workload("wide", T=1500, H=1024, I=256, E=64, k=8),
                               W.Workload("hot", T=900, H=2176, I=128, E=8, k=4),
                               W.Workload("few", T=16, H=7168, I=128, E=896, k=16)], ids=lambda w: w.name)
def test_forward_on_codes_over_many_rows(K, w):  # noqa: F811
    """Experts of both tile classes, rows longer than one step of the copy."""
    wt, p = device_weights(w), params(w)
    inp, _ = device_inputs(w)
    ids, tw = K.kmoe_route_grouped(inp["logits"], inp["bias"], w.k, n_group=4, topk_group=3)
    ids[::7, 0] = -1
    ref, _ = K.kmoe_forward(p, inp["x"], None, None, wt["w13_k"], wt["w2_k"], topk_ids=ids, topk_w=tw)
    codes, scales = K.kmoe_quantize_mx(inp["x"])
    got, ws = K.kmoe_forward_mx(p, codes, scales, ids, tw, wt["w13_k"], wt["w2_k"])
    assert K.kmoe_device_error(ws)[0] == 0
    assert torch.equal(got, ref)
