"""GPU checks that the sort, the moves, the quantisers and the block-scaled
products write their outputs and nothing beside them, whatever the tables say,
and which elements a scale that is no power of two touches."""
import numpy as np
import pytest
import torch

from tests.test_gpu_products import (BF, F32, I32, U8, K, f64, no_error, product_inputs, randn, sorted_rows)  # noqa: F401

pytestmark = pytest.mark.gpu
GUARD = 4096  # elements before and behind an output
MARK = 99     # what they and the outputs hold before


class Guarded:
    """Outputs between marks."""

    def __init__(self):
        self.held = []

    def __call__(self, *shape, dtype):
        n = int(np.prod(shape))
        flat = torch.full((2 * GUARD + n,), MARK, dtype=dtype, device="cuda")
        self.held.append((flat, n))
        return flat[GUARD:GUARD + n].view(*shape)

    def check(self):
        for flat, n in self.held:
            assert (flat[:GUARD] == MARK).all() and (flat[GUARD + n:] == MARK).all()


def live(table, M):
    """Rows that a table's segments, held inside the rows, name."""
    rows = np.zeros(M, bool)
    t = np.clip(np.array(table, np.int64), 0, M)
    for a, b in zip(t[:-1], t[1:]):
        rows[a:b] = True
    return rows


def tables(M):
    return [[0, M // 2, M // 5, 4 * M, M], [-5, 10, 2 ** 31 - 1, 30, -2 ** 31], [M] * 5, [0] * 5, [30, 40, 40, 20, 60],
            [M, M // 2, M // 4, 1, 0], [-2 ** 31, -2 ** 31, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1], [0, M, 0, M, 0]]


# few rows and many, rows shared by clusters, ends inside tiles
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("M,N,Kd", [(100, 128, 128), (100, 144, 4112), (300, 272, 144), (300, 144, 2064), (1300, 400, 400)])
def test_products_of_lying_tables(K, M, N, Kd, transpose):  # noqa: F811
    x, xs, w, ws, _ = (t if i == 4 else t.cuda() for i, t in enumerate(product_inputs(M, N, Kd, 4, transpose)))
    for to in (BF, F32):
        for table in tables(M):
            g = Guarded()
            out = g(M, Kd if transpose else N, dtype=to)
            _, work = K.kmoe_gemm_fp8(x, xs, w, ws, torch.tensor(table, dtype=I32, device="cuda"), transpose=transpose,
                                      out=out, workspace=g(256, dtype=U8)[:])
            no_error(K, work)
            g.held.pop()  # the workspace is the call's own
            g.check()
            rows = torch.from_numpy(live(table, M)).cuda()
            assert (out[~rows] == MARK).all() and (out[rows] != MARK).any(dim=1).all()


@pytest.mark.parametrize("M,N,Kd", [(100, 128, 128), (300, 272, 144), (1300, 144, 400)])
def test_columns_and_weights_gradients_of_lying_tables(K, M, N, Kd):  # noqa: F811
    E, P_ = 4, K.kmoe_fp8_padded_rows(M, 4)
    dy, x = randn(1, M, N).to(BF).cuda(), randn(2, M, Kd).to(BF).cuda()
    for table in tables(M):
        seg = torch.tensor(table, dtype=I32, device="cuda")
        g = Guarded()
        q = []
        for v in (dy, x):
            c, s = g(P_, v.shape[1], dtype=U8), g(P_ // 128, v.shape[1], dtype=F32)
            q += K.kmoe_quantize_fp8_cols(v, seg, codes=c, scales=s)
        dw = g(E, N, Kd, dtype=F32)
        _, work = K.kmoe_gemm_fp8_wgrad(*q, seg_start=seg, dw=dw)
        no_error(K, work)
        g.check()
        none = np.diff(np.clip(np.array(table, np.int64), 0, M)) <= 0
        assert (dw[torch.from_numpy(none).cuda()] == 0).all()


def test_moves_of_rows_that_are_none(K):  # noqa: F811
    for T, H, E, k in ((70, 144, 6, 3), (700, 528, 9, 4), (4100, 144, 40, 16)):
        _, row, _ = sorted_rows(T, E, k, 0.2)
        bad = row.copy()
        none = np.argwhere(row < 0)
        for (t, j), v in zip(none, [T * k, 2 ** 31 - 1, -2 ** 31, -7, T * k + 1] * len(none)):
            bad[t, j] = v
        b = torch.from_numpy(bad).cuda()
        taken = np.zeros(T * k, bool)
        taken[row[row >= 0]] = True
        free = torch.from_numpy(~taken).cuda()
        w = randn(3, T, k).cuda()
        for ty in (BF, F32):
            x, y = randn(1, T, H).to(ty).cuda(), randn(2, T * k, H).to(ty).cuda()
            g = Guarded()
            xp, out = g(T * k, H, dtype=ty), g(T, H, dtype=ty)
            d_y, d_w = g(T * k, H, dtype=ty), g(T, k, dtype=F32)
            K.kmoe_permute(x, b, out=xp)
            K.kmoe_unpermute(y, b, w, out=out)
            K.kmoe_unpermute_backward(x, y, b, w, d_y=d_y, d_w=d_w)
            g.check()
            assert (xp[free] == MARK).all() and (d_y[free] == MARK).all() and (d_w[torch.from_numpy(row < 0).cuda()] == 0).all()
        g = Guarded()
        codes, scales = g(T * k, H, dtype=U8), g(-(-H // 128), T * k, dtype=F32)
        K.kmoe_quantize_fp8(randn(1, T, H).to(BF).cuda(), b, codes=codes, scales=scales)
        g.check()
        assert (codes[free] == MARK).all() and (scales[:, free] == MARK).all()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (64, 64, 16), (65, 7, 16), (3000, 897, 7)])
def test_sort_writes_its_outputs(K, T, E, k):  # noqa: F811
    ids = torch.from_numpy(np.random.default_rng(T).integers(-3, E + 3, (T, k)).astype(np.int32)).cuda()
    g = Guarded()
    row, slot, seg = g(T, k, dtype=I32), g(T * k, dtype=I32), g(E + 1, dtype=I32)
    n = K.kmoe_sort_workspace_size(T, E, k)
    ws = torch.full((n + GUARD,), MARK, dtype=U8, device="cuda")
    K.kmoe_sort_tokens(ids, E, row_of_slot=row, slot_of_row=slot, seg_start=seg, workspace=ws)
    g.check()
    assert (ws[n:] == MARK).all()


@pytest.mark.parametrize("value", [3.0, 0.0, -1.0, float("inf"), float("nan"), 1e-40])
@pytest.mark.parametrize("rows,N,Kd,E", [(300, 272, 144, 1), (900, 144, 528, 3)])
def test_scales_that_are_no_power_of_two(K, rows, N, Kd, E, value):  # noqa: F811
    """Their row or column of the expert's weights' gradient is NaN, nothing else changes."""
    cuts = np.linspace(0, rows, E + 1).astype(np.int32)
    seg = None if E == 1 else torch.from_numpy(cuts).cuda()
    qd, qx = (K.kmoe_quantize_fp8_cols(randn(i, rows, c).to(BF).cuda(), seg) for i, c in ((1, N), (2, Kd)))
    blocks = np.concatenate([[0], np.cumsum(-(-np.diff(cuts) // 128))])
    clean, _ = K.kmoe_gemm_fp8_wgrad(*qd, *qx, seg_start=seg)
    for e in range(E):
        for of, at in ((qd, N - 1), (qd, 5), (qx, Kd - 1), (qx, 17)):
            b = blocks[e + 1] - 1
            was = float(of[1][b, at])
            of[1][b, at] = value
            dw, work = K.kmoe_gemm_fp8_wgrad(*qd, *qx, seg_start=seg)
            of[1][b, at] = was
            no_error(K, work)
            want = clean.clone()
            if of is qd:
                want[e, at] = float("nan")
            else:
                want[e, :, at] = float("nan")
            assert torch.equal(torch.isnan(dw), torch.isnan(want))
            assert torch.equal(dw.nan_to_num(0.0), want.nan_to_num(0.0))
