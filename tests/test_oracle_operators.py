"""CPU checks of the float64 definitions in oracle.operators: gradients against
central differences of the functions themselves, the grouped routing against
the plain routing and hand-made rows; and the host-side refusals of the entry
points."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import moe as O
from oracle import operators as P


def _central(f, x, dx=1e-5):
    """Gradient of the scalar f at x by central differences (error ~ dx^2)."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += dx
        b[i] -= dx
        g[i] = (f(a) - f(b)) / (2 * dx)
    return g


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(0)
    h, w, dy, d_in = rng.normal(size=(3, 7)), rng.normal(size=7), rng.normal(size=(3, 7)), rng.normal(size=(3, 7))
    dh, dw = P.rmsnorm_backward(dy, h, w, d_in, 1e-3)
    num = _central(lambda a: (P.rmsnorm(a, None, w, 1e-3)[1] * dy).sum(), h)
    assert np.allclose(dh - d_in, num, rtol=0, atol=1e-8)
    assert np.allclose(dw, _central(lambda a: (P.rmsnorm(h, None, a, 1e-3)[1] * dy).sum(), w), rtol=0, atol=1e-8)


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient_against_differences(softmax, renormalize):
    rng = np.random.default_rng(1)
    l, d_w = rng.normal(size=(4, 9)), rng.normal(size=(4, 3))
    l[1, 4] = -np.inf
    ids = np.array([[2, 0, 8], [1, 7, 3], [5, -1, 6], [-1, -1, -1]], np.int32)
    kw = dict(softmax=softmax, renormalize=renormalize, scale=2.5)
    got = P.route_backward(d_w, l, ids, **kw)
    fin = np.where(np.isneginf(l), -800.0, l)  # an expert without weight, where a difference can be taken
    assert np.allclose(got, _central(lambda a: (P.route_weights(a, ids, **kw) * d_w).sum(), fin), rtol=0, atol=1e-8)
    assert np.all(got[3] == 0)


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(2)
    T, k, H = 3, 4, 5
    y, g, w = rng.normal(size=(T * k, H)), rng.normal(size=(T, H)), rng.normal(size=(T, k))
    ids = rng.integers(0, 9, (T, k)).astype(np.int32)
    ids[1, 2], y[6] = -1, np.nan
    got = P.combine_backward(g, y, ids, 9, 2.5)
    yy = np.where(ids.reshape(-1, 1) < 0, 0.0, y)

    def loss(a):
        return (O.combine(yy.reshape(T, k, H), ids, a, 2.5) * g).sum()
    assert np.allclose(got, _central(loss, w), rtol=0, atol=1e-8)


def test_grouped_routing_without_groups_is_the_plain_routing():
    rng = np.random.default_rng(3)
    l = (rng.normal(size=(50, 96)) * 1.7).astype(np.float32)
    b = (rng.normal(size=96) * 0.1).astype(np.float32)
    ids, w = P.route_grouped(l, b, 8)
    ref, rw, _ = O.route(l, b, 8)
    assert np.array_equal(ids, ref) and np.allclose(w, rw, rtol=1e-7, atol=0)


def test_grouped_routing_by_hand():
    l = np.zeros((1, 8), np.float32)
    b = np.array([0.4, 0.0, 0.2, 0.3, 0.2, 0.2, 0.0, 0.0], np.float32)
    # groups of two: sums 1.4, 1.5, 1.4, 1.0 -> groups 1 and 0 (the lower of the equal ones)
    assert P.route_grouped(l, b, 3, n_group=4, topk_group=2)[0].tolist() == [[0, 3, 2]]
    # without a bias the logits choose, equal ones by index
    assert P.route_grouped(l, None, 3, n_group=4, topk_group=2)[0].tolist() == [[0, 1, 2]]
    l[0, 2:] = -np.inf
    ids, w = P.route_grouped(l, b, 3, n_group=4, topk_group=2)
    assert ids.tolist() == [[0, 1, -1]] and w.tolist() == [[0.5, 0.5, 0.0]]


@pytest.fixture(scope="module")
def K():
    import mxfp8_mxfp4_moe_gb300 as K
    return K


def test_norm_refusals(K):
    f = K.lib().kmoe_rmsnorm
    ok = dict(x=16, r=16, w=16, T=4, H=64, eps=1e-6, flags=0, h=16, y=16, c=16, s=16)

    def call(**kw):
        a = {**ok, **kw}
        return f(a["x"], a["r"], a["w"], a["T"], a["H"], a["eps"], a["flags"], a["h"], a["y"], a["c"], a["s"], None)
    assert call(T=-1) == 1 and call(H=0) == 1 and call(eps=-1.0) == 1 and call(eps=float("nan")) == 1
    assert call(eps=float("inf")) == 1 and call(flags=4) == 1
    assert call(x=None) == 1 and call(w=None) == 1 and call(s=None) == 1 and call(c=None) == 1
    assert call(r=None) == 1                                    # h without a residual
    assert call(h=None, y=None, c=None, s=None) == 1            # no output
    assert call(H=48) == 2 and call(H=32800) == 2               # scale groups; more columns than a block holds
    assert call(T=(1 << 30) + 1) == 2                           # more rows than 2^30
    assert call(c=8) == 3 and call(x=17) == 3 and call(r=18, flags=1) == 3 and call(w=18, flags=2) == 3
    assert call(T=0) == 0 and call(T=0, x=None, w=None) == 0    # an empty batch launches nothing


def test_norm_backward_refusals(K):
    f = K.lib().kmoe_rmsnorm_backward
    n = K.kmoe_rmsnorm_workspace_size(4, 64)
    assert n > 0 and K.kmoe_rmsnorm_workspace_size(-1, 64) == 0 and K.kmoe_rmsnorm_workspace_size(4, 0) == 0
    assert K.kmoe_rmsnorm_workspace_size(4, 32800) == 0 and K.kmoe_rmsnorm_workspace_size((1 << 30) + 1, 64) == 0
    ok = dict(dy=16, h=16, w=16, di=16, T=4, H=64, eps=1e-6, flags=0, dh=16, dw=16, ws=256, n=n)

    def call(**kw):
        a = {**ok, **kw}
        return f(a["dy"], a["h"], a["w"], a["di"], a["T"], a["H"], a["eps"], a["flags"], a["dh"], a["dw"], a["ws"],
                 a["n"], None)
    assert call(T=-1) == 1 and call(H=0) == 1 and call(eps=-1.0) == 1 and call(flags=8) == 1 and call(H=32800) == 2
    assert call(dy=None) == 1 and call(h=None) == 1 and call(w=None) == 1 and call(dh=None) == 1
    assert call(dw=None) == 1 and call(T=0, dw=None) == 1
    assert call(ws=None) == 5 and call(n=n - 1) == 5 and call(ws=128) == 3
    assert call(dh=17) == 3 and call(di=18, flags=1) == 3 and call(dw=18) == 3


def test_route_refusals(K):
    P_ = K.kmoe_route_params
    ok = dict(T=4, E=16, k=4, n_group=4, topk_group=2, flags=0, scale=1.0)
    for f in (K.lib().kmoe_route_grouped, K.lib().kmoe_route_backward):
        def call(a=16, b=16, c=16, d=16, **kw):
            return f(ctypes.byref(P_(*{**ok, **kw}.values())), a, b, c, d, None)
        assert f(None, 16, 16, 16, 16, None) == 1
        assert call(T=-1) == 1 and call(E=0) == 1 and call(E=1028) == 1 and call(k=0) == 1 and call(k=17) == 1
        assert call(E=64, k=33, topk_group=4) == 1                      # more slots than a token can have
        assert call(n_group=0) == 1 and call(n_group=64, E=64) == 1 and call(topk_group=0) == 1
        assert call(topk_group=5) == 1 and call(flags=4) == 1 and call(scale=float("nan")) == 1
        assert call(scale=float("inf")) == 1
        assert call(E=18) == 2 and call(k=9) == 2                       # unequal groups; fewer experts than slots
        assert call(T=(1 << 28) + 1) == 2                               # more slots than 2^30
        assert call(a=None) == 1 and call(c=None) == 1 and call(d=None) == 1
        assert call(a=18) == 3 and call(d=18) == 3
        assert call(T=0, a=None, b=None, c=None, d=None) == 0


def test_combine_backward_and_forward_mx_refusals(K):
    f = K.lib().kmoe_combine_backward
    assert f(16, 16, 16, -1, 64, 2, 8, 1.0, 16, None) == 1 and f(16, 16, 16, 4, 0, 2, 8, 1.0, 16, None) == 1
    assert f(16, 16, 16, 4, 64, 9, 8, 1.0, 16, None) == 1 and f(16, 16, 16, 4, 64, 2, 2000, 1.0, 16, None) == 1
    assert f(16, 16, 16, 4, 66, 2, 8, 1.0, 16, None) == 2 and f(16, 16, 16, 1 << 30, 64, 2, 8, 1.0, 16, None) == 2
    assert f(None, 16, 16, 4, 64, 2, 8, 1.0, 16, None) == 1 and f(16, 16, 16, 4, 64, 2, 8, 1.0, None, None) == 1
    assert f(16, 8, 16, 4, 64, 2, 8, 1.0, 16, None) == 3 and f(4, 16, 16, 4, 64, 2, 8, 1.0, 16, None) == 3
    assert f(None, None, None, 0, 64, 2, 8, 1.0, None, None) == 0
    p = K.make_params(16, 128, 128, 8, 2)
    n = K.kmoe_workspace_size(p)
    g = K.lib().kmoe_forward_mx
    assert g(None, 16, 16, 16, 16, 256, 256, 16, 256, n, None) == 1
    assert g(ctypes.byref(p), None, 16, 16, 16, 256, 256, 16, 256, n, None) == 1
    assert g(ctypes.byref(p), 16, None, 16, 16, 256, 256, 16, 256, n, None) == 1
    assert g(ctypes.byref(p), 16, 16, None, 16, 256, 256, 16, 256, n, None) == 1
    assert g(ctypes.byref(p), 16, 16, 16, None, 256, 256, 16, 256, n, None) == 1
    assert g(ctypes.byref(p), 8, 16, 16, 16, 256, 256, 16, 256, n, None) == 3
    assert g(ctypes.byref(p), 16, 18, 16, 16, 256, 256, 16, 256, n, None) == 3
    assert g(ctypes.byref(p), 16, 16, 16, 16, 256, 256, 16, 256, n - 1, None) == 5


def test_binding_refusals(K):
    bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8

    def rejects(fn, needle):
        with pytest.raises(ValueError, match=needle):
            fn()
    x, w = torch.zeros(4, 64, dtype=bf), torch.zeros(64)
    rejects(lambda: K.kmoe_rmsnorm(x, torch.zeros(63)), r"weight must have shape \(64,\)")
    rejects(lambda: K.kmoe_rmsnorm(x, w.half()), "weight must be torch.bfloat16 or torch.float32")
    rejects(lambda: K.kmoe_rmsnorm(x.float(), w), "x must be torch.bfloat16")
    rejects(lambda: K.kmoe_rmsnorm(x[0], w), "2-D")
    rejects(lambda: K.kmoe_rmsnorm(x, w, residual=torch.zeros(4, 64), h=x), "h must be torch.float32")
    rejects(lambda: K.kmoe_rmsnorm(x, w, h=x), "needs a residual")
    rejects(lambda: K.kmoe_rmsnorm(x, w, codes=torch.zeros(4, 64, dtype=u8)), "need mx=True")
    rejects(lambda: K.kmoe_rmsnorm(x, w, mx=True, scales=torch.zeros(4, 1, dtype=u8)), "scales must have shape")
    rejects(lambda: K.kmoe_rmsnorm(torch.zeros(64, 4, dtype=bf).t(), w), "contiguous")
    rejects(lambda: K.kmoe_rmsnorm(x, w), "CUDA tensor")
    rejects(lambda: K.kmoe_rmsnorm_backward(x.float(), x, w), "dy must be torch.bfloat16")
    rejects(lambda: K.kmoe_rmsnorm_backward(x, x.float(), w, dh_in=x), "dh_in must be torch.float32")
    rejects(lambda: K.kmoe_rmsnorm_backward(x, x, w, dweight=torch.zeros(64, dtype=bf)), "dweight must be")
    lg, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=i32)
    rejects(lambda: K.kmoe_route_grouped(lg, torch.zeros(7), 2), "bias must have shape")
    rejects(lambda: K.kmoe_route_grouped(lg, None, 2, topk_w=torch.zeros(4, 3)), "topk_w must have shape")
    rejects(lambda: K.kmoe_route_grouped(lg.double(), None, 2), "logits must be torch.float32")
    rejects(lambda: K.kmoe_route_grouped(lg, None, 2), "CUDA tensor")
    rejects(lambda: K.kmoe_route_backward(torch.zeros(4, 3), lg, ids), "d_w must have shape")
    rejects(lambda: K.kmoe_route_backward(torch.zeros(4, 2), lg, ids, d_logits=torch.zeros(4, 7)), "d_logits")
    rejects(lambda: K.kmoe_combine_backward(x, torch.zeros(7, 64), ids, 8), r"y must have shape \(8, 64\)")
    p = K.make_params(4, 128, 128, 8, 2)
    q, sc = torch.zeros(4, 128, dtype=u8), torch.zeros(4, 4, dtype=u8)
    rejects(lambda: K.kmoe_forward_mx(p, q[:, :64], sc, ids, lg[:, :2], q, q), "x_codes must have shape")
    rejects(lambda: K.kmoe_forward_mx(p, q, sc[:3], ids, lg[:, :2], q, q), "x_scales must have shape")
    rejects(lambda: K.kmoe_forward_mx(p, q, sc, ids.long(), lg[:, :2].contiguous(), q, q), "topk_ids must be")
