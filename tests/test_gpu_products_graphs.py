"""GPU checks of the sort and the quantisation, whose scratch memory is their own,
in captured graphs, and of the block-scaled products at the ends of their sizes."""
import numpy as np
import pytest
import torch

from oracle import products as P
from tests.test_gpu_products import (BF, F32, K, no_error, product_inputs, product_tolerance, randn, routing,  # noqa: F401
                                     within)

pytestmark = pytest.mark.gpu


def test_graphs_that_live_together_keep_their_scratch(K):  # noqa: F811
    """Two captured, replayed with other inputs between other allocations, in turn and at once."""
    T, E, k, H = 4200, 40, 16, 144
    assert K.kmoe_quantize_fp8_workspace_size(T, H, k) > 0

    def inputs(seed):
        return torch.from_numpy(routing(seed, T, E, k, 0.1)).cuda(), randn(seed, T, H).to(BF).cuda()

    def chain(ids, x):
        row, slot, seg = K.kmoe_sort_tokens(ids, E)
        codes, scales = K.kmoe_quantize_fp8(x, row)
        live = torch.arange(T * k, device="cuda") < seg[-1]
        return row, slot, seg, torch.where(live[:, None], codes, 0), torch.where(live, scales, 0.0)

    want = [[t.clone() for t in chain(*inputs(s))] for s in (3, 4)]
    held, graphs = [inputs(1), inputs(2)], []
    torch.cuda.synchronize()
    for given in held:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = chain(*given)
        graphs.append((g, out))
    for given, seed in zip(held, (3, 4)):
        for t, other in zip(given, inputs(seed)):
            t.copy_(other)

    def check():
        torch.cuda.synchronize()
        for (_, out), ref in zip(graphs, want):
            for a, b in zip(out, ref):
                assert torch.equal(a, b)
                a.zero_()

    for _ in range(3):
        for g, _ in graphs:
            g.replay()
            junk = [torch.full((1 << 18,), 255, device="cuda") for _ in range(8)]
        del junk
    check()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    check()


ENDS = [(1, 16, 16, 1024, None), (1024, 16, 16, 1024, None), (33, 16, 1 << 17, 1, None), (1, 1 << 17, 16, 1, None),
        (300, 16, 16, 2, None), (257, 1 << 16, 16, 1, None), (20000, 16, 32, 1024, None), (700, 272, 400, 3, [0, 0, 700]),
        (60, 272, 400, 1, [50]), (600, 272, 400, 1, [333])]


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("M,N,Kd,E,counts", ENDS)
def test_products_at_the_ends_of_their_sizes_on_a_stream(K, M, N, Kd, E, counts, transpose):  # noqa: F811
    x, xs, w, ws, seg = product_inputs(M, N, Kd, E, transpose)
    if counts is not None:  # (also one expert with rows behind its last)
        seg = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    ref, mag = P.gemm(P.values_rows(x.numpy(), xs.numpy()), P.values_weights(w.numpy(), ws.numpy()), seg, transpose)
    out = torch.full(ref.shape, float("nan"), device="cuda")
    args = [t.cuda() for t in (x, xs, w, ws)]
    table = None if E == 1 and counts is None else torch.from_numpy(seg).cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    _, work = K.kmoe_gemm_fp8(*args, table, transpose=transpose, out=out, stream=side)
    side.synchronize()
    no_error(K, work)
    within(out, ref, product_tolerance(ref, mag, N if transpose else Kd, F32), "out")
