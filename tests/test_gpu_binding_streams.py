"""Calls on a stream of their own while the current stream still uses memory that its tensors had."""
import pytest
import torch

from tests._moe_setup import device_inputs, device_weights, params
from tests.test_gpu_operators import BF, K, randn  # noqa: F401
import workloads as W

pytestmark = pytest.mark.gpu


def test_outputs_do_not_take_memory_in_use(K):  # noqa: F811
    """The current stream has yet to read tensors of every output's size that
    the caller has let go of; the calls run at once on another stream."""
    T, H, E, k = 512, 1024, 256, 8
    x, r, nw = randn(1, T, H).to(BF).cuda(), randn(2, T, H).to(BF).cuda(), randn(3, H).cuda()
    lg, d_w, y3, bias = (t.cuda() for t in (randn(4, T, E), randn(5, T, k), randn(6, T * k, H), randn(7, E)))
    w = W.WORKLOADS["tiny"]
    wt, p = device_weights(w), params(w)
    inp, _ = device_inputs(w)
    codes, scales = K.kmoe_quantize_mx(inp["x"])

    def layer(stream):
        ids, tw = K.kmoe_route(inp["logits"], inp["bias"], w.k, stream=stream)
        a, wa = K.kmoe_forward(p, inp["x"], inp["logits"], inp["bias"], wt["w13_k"], wt["w2_k"], stream=stream)
        b, wb = K.kmoe_forward_mx(p, codes, scales, ids, tw, wt["w13_k"], wt["w2_k"], stream=stream)
        return [ids, tw, a, b, *K.kmoe_quantize_mx(x, stream=stream)], [wa, wb]

    def calls(stream=None):
        h, y, c, s = K.kmoe_rmsnorm(x, nw, residual=r, mx=True, stream=stream)
        ids, tw = K.kmoe_route_grouped(lg, bias, k, n_group=8, topk_group=4, stream=stream)
        out, ws = layer(stream)
        return [h, y, c, s, ids, tw, K.kmoe_route_backward(d_w, lg, ids, stream=stream),
                K.kmoe_combine_backward(x, y3, ids, E, stream=stream),
                *K.kmoe_rmsnorm_backward(y, h, nw, dh_in=x, stream=stream), *out], ws
    ref, ws = calls()
    ref = [t.clone() for t in ref]
    side = torch.cuda.Stream()
    victims = [torch.empty_like(t).view(torch.uint8).fill_(7) for t in ref + ws]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some tens of milliseconds
    read = [t.clone() for t in victims]
    del victims, ws
    got, _ = calls(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in read)


def test_inputs_are_kept_until_their_stream_is_through(K):  # noqa: F811
    """The caller lets go of its inputs while the other stream has yet to read them."""
    T, E, k, H = 256, 256, 8, 1024
    lg, bias = randn(1, T, E).cuda(), randn(2, E).cuda()
    x = randn(3, T, H).to(BF).cuda()
    ref = (*K.kmoe_route(lg, bias, k), *K.kmoe_quantize_mx(x))
    side = torch.cuda.Stream()
    for _ in range(3):
        a, b, c = lg.clone(), bias.clone(), x.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = (*K.kmoe_route(a, b, k, stream=side), *K.kmoe_quantize_mx(c, stream=side))
        del a, b, c
        again = [torch.full_like(t, float("nan")) for t in (lg, bias, x)]  # what the allocator hands out next
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(ref, got))
        del again
