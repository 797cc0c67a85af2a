"""The gradient of renormalised softmax weights where the row's largest logit
is not among the chosen ones: the weights count a score below e^-700 of the
largest as 0, wherever on the axis the row lies, and so does their gradient."""
import numpy as np
import pytest
import torch

from oracle import operators as P
from tests.test_gpu_operators import K, at_offset, check_route, check_route_gradient, randn  # noqa: F401

pytestmark = pytest.mark.gpu
FORCED = [3, 17, 30, 41]  # chosen by their bias


def rows_below_a_top(T, E):
    """Rows whose top logit stands at 7, far above the chosen ones or not."""
    logits, bias = 1.7 * randn(1, T, E), 0.1 * randn(2, E)
    bias[FORCED] = 5.0
    special = [(500.0, [-199.9, -200.1, -199.95, -250.0]), (500.0, [-250.0, -249.0, -251.0, -250.5]),
               (1e4, [0.0, 1.0, 2.0, 3.0]), (float("inf"), [0.0, -1.0, 1.0, 2.0]), (3e38, [1e30, 0.0, 1.0, 5.0]),
               (1e4, [9301.0, 9299.0, 9300.5, 9400.0]), (2.0, [-690.0, -699.0, -1.0, -400.0])]
    for i, (top, chosen) in enumerate(special):
        for t in range(i, T, len(special) + 1):  # every eighth row is an ordinary one
            logits[t, 7] = top
            logits[t, FORCED] = torch.tensor(chosen)
    return logits, bias


@pytest.mark.parametrize("T,E", [(8, 48), (8, 897), (700, 896), (11, 1024)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_under_a_distant_top(K, T, E, renormalize):  # noqa: F811
    logits, bias = rows_below_a_top(T, E)
    ids, w = check_route(K, logits, bias, 4, 1, 1, True, renormalize, 2.5)
    n = ids.cpu().numpy()
    assert (np.sort(n, axis=1) == FORCED).all()
    d_w = randn(3, T, 4)
    ref = P.route_backward(d_w.double().numpy(), logits.numpy(), n, True, renormalize, 2.5)
    for lg in (logits.cuda(), at_offset(logits, 1)):
        got = K.kmoe_route_backward(d_w.cuda(), lg, ids, score="softmax", renormalize=renormalize, scale=2.5)
        check_route_gradient(got, ref, d_w.double().numpy(), logits, n, True, renormalize, 2.5)
    # what weighs nothing has no gradient
    assert not got[1, n[1]].any() and not got[3, n[3]].any()


def test_route_gradient_does_not_move_with_the_row(K):  # noqa: F811
    """A constant added to a row (exactly: the logits lie on a grid of 1/64) changes no weight and no gradient."""
    T, E = 5, 48
    logits, bias = torch.round(64 * 1.7 * randn(1, T, E)) / 64, 0.1 * randn(2, E)
    bias[FORCED] = 5.0
    logits[:, 7] = 500.0
    logits[:, FORCED] = torch.tensor([[-198.0, -200.0, -201.0, -199.5], [-250.0, -249.0, -251.0, -250.5],
                                      [300.0, 301.0, -202.0, 299.0], [-100.0, -200.5, -150.0, -201.0],
                                      [499.0, 498.0, 497.0, -300.0]])
    d_w = randn(4, T, 4).cuda()
    ids, w = K.kmoe_route_grouped(logits.cuda(), bias.cuda(), 4, score="softmax")
    ref = K.kmoe_route_backward(d_w, logits.cuda(), ids, score="softmax")
    for shift in (-1024.0, 1024.0):
        moved = (logits + shift).cuda()
        assert torch.equal(K.kmoe_route_grouped(moved, bias.cuda(), 4, score="softmax")[1], w)
        assert torch.equal(K.kmoe_route_backward(d_w, moved, ids, score="softmax"), ref)
