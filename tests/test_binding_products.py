"""How the binding of the sort and the block-scaled products treats streams and
GPUs, on the CPU, against the stand-ins of test_binding_streams."""
import pytest
import torch

import mxfp8_mxfp4_moe_gb300 as K
from tests.test_binding_streams import BF, F32, I32, U8, Tensor, gpu  # noqa: F401  (gpu: a fixture)


def calls():
    """(name, tensors it is given, call) of every entry point that launches."""
    T, k, E, N, Kd, H = 4, 2, 3, 64, 144, 64
    R, P = T * k, K.kmoe_fp8_padded_rows(T * k, E)
    rows, seg = ((T, k), I32), ((E + 1,), I32)
    row = []

    def add(fn, post=(), **kw):
        t = {n: Tensor(s, d) for n, (s, d) in kw.items()}
        row.append((fn.__name__, t, lambda **o: fn(**t, **dict(post), **o)))
    add(K.kmoe_sort_tokens, topk_ids=rows, post=dict(E=E))
    add(K.kmoe_permute, x=((T, H), BF), row_of_slot=rows)
    add(K.kmoe_unpermute, y=((R, H), F32), row_of_slot=rows, topk_w=((T, k), F32))
    add(K.kmoe_unpermute_backward, d_out=((T, H), BF), y=((R, H), BF), row_of_slot=rows, topk_w=((T, k), F32))
    add(K.kmoe_quantize_fp8, x=((T, H), BF), row_of_slot=rows)
    add(K.kmoe_quantize_fp8_weights, w=((E, N, Kd), BF))
    add(K.kmoe_quantize_fp8_cols, x=((R, Kd), BF), seg_start=seg)
    add(K.kmoe_gemm_fp8, x=((R, Kd), U8), x_scales=((2, R), F32), w=((E, N, Kd), U8), w_scales=((E, 1, 2), F32),
        seg_start=seg)
    add(K.kmoe_gemm_fp8_wgrad, dy=((P, N), U8), dy_scales=((P // 128, N), F32), x=((P, Kd), U8),
        x_scales=((P // 128, Kd), F32), seg_start=seg)
    return row


NAMES = [c[0] for c in calls()]


def named(name):
    return dict((c[0], c[1:]) for c in calls())[name]


@pytest.fixture
def box(gpu, monkeypatch):  # noqa: F811
    real = gpu.lib.real
    monkeypatch.setattr(type(gpu.lib), "kmoe_fp8_padded_rows", property(lambda self: real.kmoe_fp8_padded_rows),
                        raising=False)
    return gpu


def test_every_launching_entry_point_is_here():
    assert set(NAMES) == {n for n in K.PRODUCT_EXPORTS if not n.endswith(("_size", "_padded_rows"))}


@pytest.mark.parametrize("name", NAMES)
def test_outputs_come_from_the_streams_own_memory(box, name):
    given, fn = named(name)
    fn(stream=box.side)
    assert box.made and all(t.pool is box.side for t in box.made) and all(box.current in t.used_by for t in box.made)
    assert box.lib.launched and all(handle == box.side.cuda_stream for _, handle in box.lib.launched)
    assert all(handle == box.side.cuda_stream for handle in box.scratch)
    assert all(box.side in t.used_by for t in given.values())


@pytest.mark.parametrize("name", NAMES)
def test_without_a_stream_calls_use_the_current_one(box, name):
    named(name)[1]()
    assert box.made and all(t.pool is box.current and not t.used_by for t in box.made)
    assert box.lib.launched and all(handle == box.current.cuda_stream for _, handle in box.lib.launched)


@pytest.mark.parametrize("name", NAMES)
def test_tensors_on_another_gpu_are_refused(box, name):
    given, fn = named(name)
    box.device = 1
    with pytest.raises(ValueError, match=r"on cuda:0.*cuda:1"):
        fn()
    box.device = 0
    for t in given.values():
        t.index, t.device = 1, torch.device("cuda", 1)
        with pytest.raises(ValueError, match="on cuda:"):
            fn()
        t.index, t.device = 0, torch.device("cuda", 0)
    box.side.device_index, box.side.device = 1, torch.device("cuda", 1)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        fn(stream=box.side)
    assert not box.made and not box.lib.launched and not box.scratch


def test_workspaces_that_are_given_are_checked_and_held(box):
    n = {"kmoe_sort_tokens": K.kmoe_sort_workspace_size(4, 3, 2), "kmoe_quantize_fp8": 1}
    for name in ("kmoe_sort_tokens", "kmoe_quantize_fp8", "kmoe_gemm_fp8", "kmoe_gemm_fp8_wgrad"):
        fn, size = named(name)[1], max(n.get(name, 256), 1)
        with pytest.raises(ValueError, match="workspace is on cuda:1"):
            fn(workspace=Tensor((size,), U8, 1))
        ws = Tensor((size,), U8)
        fn(workspace=ws, stream=box.side)
        assert box.side in ws.used_by
    assert not box.scratch


def test_many_rows_take_scratch_for_their_scales(box):
    T, k = 4096, 16
    K.kmoe_quantize_fp8(Tensor((T, 64), BF), Tensor((T, k), I32))
    assert box.scratch == [box.current.cuda_stream]
