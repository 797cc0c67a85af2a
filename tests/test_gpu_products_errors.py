"""GPU checks of the device error word of the block-scaled products' workspaces."""
import pytest
import torch

from tests.test_gpu_products import BF, F32, I32, U8, K, no_error, randn  # noqa: F401 (K: a fixture)

pytestmark = pytest.mark.gpu


def product(K, M, **kw):  # noqa: F811
    N, Kd = 128, 256
    e = lambda *s, dtype=U8: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    return K.kmoe_gemm_fp8(e(M, Kd), e(Kd // 128, M, dtype=F32), e(N, Kd), e(1, Kd // 128, dtype=F32), **kw)[1]


def dirty(stream=None):
    """Memory of a workspace's size, all ones, back in the allocator's hands."""
    with torch.cuda.stream(stream):
        for t in [torch.full((K_BYTES,), 255, dtype=U8, device="cuda") for _ in range(64)]:
            del t
    torch.cuda.synchronize()


K_BYTES = 256


def test_a_call_without_rows_has_no_error(K):  # noqa: F811
    side = torch.cuda.Stream()
    for stream in (None, side):
        held = []
        for _ in range(40):
            dirty(stream)
            held.append(product(K, 0, stream=stream))
        torch.cuda.synchronize()
        for work in held:
            no_error(K, work)


def test_the_word_stays_until_the_next_product_in_its_workspace(K):  # noqa: F811
    work = torch.full((K_BYTES,), 0, dtype=U8, device="cuda")
    work[0] = 1
    product(K, 0, workspace=work)
    product(K, 4)
    assert K.kmoe_device_error(work) == (7, 1)  # KMOE_ERR_TIMEOUT, as a wait that ran out leaves it; reading clears it
    no_error(K, work)
    work[0] = 1
    product(K, 4, workspace=work)
    no_error(K, work)
    work[0] = 1
    product(K, 300, workspace=work)
    no_error(K, work)
    for P_ in (0, 128):
        work[0] = 1
        z = [torch.zeros(P_, c, dtype=U8, device="cuda") for c in (128, 256)]
        s = [torch.ones(P_ // 128, c, device="cuda") for c in (128, 256)]
        K.kmoe_gemm_fp8_wgrad(z[0], s[0], z[1], s[1], workspace=work)
        no_error(K, work)


def test_each_product_of_a_layer_reports(K):  # noqa: F811
    """Forward, the rows' gradient and the weights', each in a workspace of its own."""
    T, E, k, N, Kd = 60, 5, 2, 272, 400
    x, g = randn(1, T, Kd).to(BF).cuda(), randn(2, T, N).to(BF).cuda()
    ids = (torch.arange(T * k, dtype=I32, device="cuda") * 7 % E).view(T, k)
    w, ws = K.kmoe_quantize_fp8_weights(randn(3, E, N, Kd).to(BF).cuda())
    row, _, seg = K.kmoe_sort_tokens(ids, E)
    y, w1 = K.kmoe_gemm_fp8(*K.kmoe_quantize_fp8(x, row), w, ws, seg)
    d_y, _ = K.kmoe_unpermute_backward(g, y, row, torch.ones(T, k, device="cuda"))
    _, w2 = K.kmoe_gemm_fp8(*K.kmoe_quantize_fp8(d_y), w, ws, seg, transpose=True)
    _, w3 = K.kmoe_gemm_fp8_wgrad(*K.kmoe_quantize_fp8_cols(d_y, seg),
                                  *K.kmoe_quantize_fp8_cols(K.kmoe_permute(x, row), seg), seg_start=seg)
    assert len({t.data_ptr() for t in (w1, w2, w3)}) == 3
    for work in (w1, w2, w3):
        no_error(K, work)
