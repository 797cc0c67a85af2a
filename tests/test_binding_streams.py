"""How the binding treats streams, on the CPU: every call runs against stand-ins
for the library's launches, CUDA tensors, streams and the caching allocator."""
import contextlib
import types

import pytest
import torch

import mxfp8_mxfp4_moe_gb300 as K

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class Tensor:
    """A CUDA tensor as far as the binding looks at one."""
    count = 0

    def __init__(self, shape, dtype, device=0, pool=None):
        Tensor.count += 1
        self.shape = torch.Size(shape if isinstance(shape, (tuple, list, torch.Size)) else (shape,))
        self.dtype, self.index, self.pool, self.used_by = dtype, device, pool, []
        self.device, self.is_cuda, self.at = torch.device("cuda", device), True, 4096 * Tensor.count

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.index

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at

    def record_stream(self, stream):
        self.used_by.append(stream)


class Library:
    """The library with launches that only note their last argument, the stream."""

    def __init__(self, real):
        self.real, self.launched = real, []

    def __getattr__(self, name):
        if name.endswith(("_size", "_bytes", "_string", "_layout")):
            return getattr(self.real, name)

        def launch(*args):
            ev = name in ("kmoe_forward_ex", "kmoe_forward_router")  # the events come last there
            handle = args[-2] if ev else args[-1]
            self.launched.append((name, getattr(handle, "value", handle)))
            return 0
        return launch


@pytest.fixture
def gpu(monkeypatch):
    """A stand-in GPU: `current` and `side` streams, the current device, and the allocations made."""
    box = types.SimpleNamespace(device=0, made=[], scratch=[], lib=Library(K._lib))
    box.current = types.SimpleNamespace(cuda_stream=0x70, device_index=0, device=torch.device("cuda", 0))
    box.side = types.SimpleNamespace(cuda_stream=0x90, device_index=0, device=torch.device("cuda", 0))
    box.stream = box.current

    def empty(shape, dtype=None, device=None, **kw):
        index = device if isinstance(device, int) else torch.device(device).index
        t = Tensor(shape, dtype, index, box.stream)
        box.made.append(t)
        return t

    @contextlib.contextmanager
    def on(stream):
        before, box.stream = box.stream, stream
        yield
        box.stream = before

    def alloc(size, handle):
        box.scratch.append(handle)
        return 1 << 20
    driver = {"_cuda_getCurrentRawStream": lambda dev: box.stream.cuda_stream, "_cuda_getDevice": lambda: box.device,
              "_cuda_cudaCachingAllocator_raw_alloc": alloc, "_cuda_cudaCachingAllocator_raw_delete": lambda at: None}
    for name, fn in driver.items():
        monkeypatch.setattr(torch._C, name, fn, raising=False)
    # what the package bound of them when it was imported
    for name, of in (("_current_stream", "_cuda_getCurrentRawStream"), ("_current_device", "_cuda_getDevice"),
                     ("_scratch_alloc", "_cuda_cudaCachingAllocator_raw_alloc"),
                     ("_scratch_free", "_cuda_cudaCachingAllocator_raw_delete")):
        if hasattr(K, name):
            monkeypatch.setattr(K, name, driver[of])
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", lambda t: empty(t.shape, t.dtype, t.device))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: box.stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: box.device)
    monkeypatch.setattr(K, "_lib", box.lib)
    return box


def calls(device=0):
    """(name, tensors it is given, call) of every entry point that launches."""
    T, H, I, E, k = 4, 128, 128, 8, 2
    p = K.make_params(T, H, I, E, k)

    def given(**kw):
        return {n: Tensor(s, d, device) for n, (s, d) in kw.items()}
    x, lg, w = ((T, H), BF), ((T, E), F32), ((T, k), F32)
    ids, bias = ((T, k), I32), ((E,), F32)
    w13, w2 = ((K.kmoe_prepared_weight_bytes(p, 0),), U8), ((K.kmoe_prepared_weight_bytes(p, 1),), U8)
    layer = dict(x=x, logits=lg, bias=bias, w13_k=w13, w2_k=w2)
    row = []

    def add(fn, args=(), pre=(), post=(), **kw):
        t = given(**kw)
        row.append((fn.__name__, t, lambda **o: fn(*pre, **t, **dict(post), **o)))
    add(K.kmoe_route, logits=lg, bias=bias, post=dict(k=k))
    add(K.kmoe_quantize_mx, x=x)
    add(K.kmoe_prepare_weights, pre=(p,), w13=((E, 2 * I, H // 2), U8), w13_sf=((E, 2 * I, H // 32), U8),
        w2=((E, H, I // 2), U8), w2_sf=((E, H, I // 32), U8))
    add(K.kmoe_forward, pre=(p,), **layer)
    add(K.kmoe_router, x=x, w_gate=((E, H), BF), bias=bias, post=dict(k=k))
    add(K.kmoe_forward_router, pre=(p,), x=x, w_gate=((E, H), BF), bias=bias, w13_k=w13, w2_k=w2)
    add(K.kmoe_forward_noalloc, pre=(p,), **layer)
    add(K.kmoe_selftest_activation, pre=(p,), gate=((5,), F32), up=((5,), F32))
    add(K.kmoe_forward_mx, pre=(p,), x_codes=((T, H), U8), x_scales=((T, H // 32), U8), topk_ids=ids, topk_w=w,
        w13_k=w13, w2_k=w2)
    add(K.kmoe_rmsnorm, x=x, weight=((H,), F32), residual=x, post=dict(mx=True))
    add(K.kmoe_rmsnorm_backward, dy=x, h=x, weight=((H,), F32), dh_in=x)
    add(K.kmoe_route_grouped, logits=lg, bias=bias, post=dict(k=k))
    add(K.kmoe_route_backward, d_w=w, logits=lg, topk_ids=ids)
    add(K.kmoe_combine_backward, d_out=x, y=((T * k, H), F32), topk_ids=ids, post=dict(E=E))
    return row


NAMES = [c[0] for c in calls()]


def test_every_launching_entry_point_is_here():
    plain = {"kmoe_status_string", "kmoe_check_device", "kmoe_workspace_size", "kmoe_workspace_layout",
             "kmoe_prepared_weight_bytes", "kmoe_tile_sf_offset", "kmoe_router_workspace_size",
             "kmoe_rmsnorm_workspace_size"}
    no_tensors_of_their_own = {"kmoe_forward_ex", "kmoe_device_error", "kmoe_selftest_wait_timeout",
                               "kmoe_mma_peak_run"}
    assert set(NAMES) == set(K.EXPORTS) - plain - no_tensors_of_their_own


@pytest.mark.parametrize("name", NAMES)
def test_outputs_come_from_the_streams_own_memory(gpu, name):
    """What a call on a given stream allocates is that stream's memory: a block
    that the caller's stream is not through with is not handed out; and the
    caller's stream, which goes on with the outputs, holds them too."""
    fn = dict((c[0], c[2]) for c in calls())[name]
    fn(stream=gpu.side)
    assert gpu.made and all(t.pool is gpu.side for t in gpu.made)
    assert all(gpu.current in t.used_by for t in gpu.made)
    assert all(handle == gpu.side.cuda_stream for _, handle in gpu.lib.launched) and gpu.lib.launched
    assert all(handle == gpu.side.cuda_stream for handle in gpu.scratch)
    assert gpu.stream is gpu.current


@pytest.mark.parametrize("name", NAMES)
def test_without_a_stream_calls_use_the_current_one(gpu, name):
    fn = dict((c[0], c[2]) for c in calls())[name]
    fn()
    assert gpu.made and all(t.pool is gpu.current and not t.used_by for t in gpu.made)
    assert all(handle == gpu.current.cuda_stream for _, handle in gpu.lib.launched) and gpu.lib.launched


@pytest.mark.parametrize("name", NAMES)
def test_tensors_are_held_for_the_stream_that_uses_them(gpu, name):
    """The caller's tensors are kept from reuse until the given stream is through with them."""
    given, fn = dict((c[0], c[1:]) for c in calls())[name]
    fn(stream=gpu.side)
    assert all(gpu.side in t.used_by for t in given.values())


@pytest.mark.parametrize("fn", [K.kmoe_device_error, lambda ws, stream: K.kmoe_mma_peak_run(1, 64, ws, stream),
                                lambda ws, stream: K.kmoe_selftest_wait_timeout(ws, 1, stream)])
def test_workspaces_are_held_too(gpu, monkeypatch, fn):
    monkeypatch.setattr(torch.cuda, "get_device_properties",
                        lambda dev: types.SimpleNamespace(multi_processor_count=152))
    ws = Tensor((4096,), U8)
    fn(ws, stream=gpu.side)
    assert gpu.side in ws.used_by


def test_outputs_that_are_given_are_held(gpu):
    x, w = Tensor((4, 128), BF), Tensor((128,), F32)
    out = [Tensor((4, 128), BF), Tensor((128,), F32), Tensor((K.kmoe_rmsnorm_workspace_size(4, 128),), U8)]
    K.kmoe_rmsnorm_backward(x, x, w, dh=out[0], dweight=out[1], workspace=out[2], stream=gpu.side)
    q = [Tensor((4, 128), U8), Tensor((4, 4), U8)]
    K.kmoe_quantize_mx(x, codes=q[0], scales=q[1], stream=gpu.side)
    assert all(gpu.side in t.used_by for t in out + q)


@pytest.mark.parametrize("name", NAMES)
def test_tensors_on_another_gpu_are_refused(gpu, name):
    """Launches go to the current GPU: tensors or a stream of another are refused before anything is allocated."""
    given, fn = dict((c[0], c[1:]) for c in calls())[name]
    gpu.device = 1
    with pytest.raises(ValueError, match=r"on cuda:0.*cuda:1"):
        fn()
    gpu.device = 0
    for arg, t in given.items():
        t.index, t.device = 1, torch.device("cuda", 1)
        with pytest.raises(ValueError, match="on cuda:"):
            fn()
        t.index, t.device = 0, torch.device("cuda", 0)
    gpu.side.device_index, gpu.side.device = 1, torch.device("cuda", 1)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        fn(stream=gpu.side)
    assert not gpu.made and not gpu.lib.launched and not gpu.scratch
    fn()
    assert gpu.lib.launched


def test_outputs_and_workspaces_on_another_gpu_are_refused(gpu):
    x, w = Tensor((4, 128), BF), Tensor((128,), F32)
    n = K.kmoe_rmsnorm_workspace_size(4, 128)
    far = dict(dh=Tensor((4, 128), BF, 1), dweight=Tensor((128,), F32, 1), workspace=Tensor((n,), U8, 1))
    for arg, t in far.items():
        with pytest.raises(ValueError, match=f"{arg} is on cuda:1"):
            K.kmoe_rmsnorm_backward(x, x, w, **{arg: t})
    given, fn = dict((c[0], c[1:]) for c in calls())["kmoe_forward_mx"]
    with pytest.raises(ValueError, match="workspace is on cuda:1"):
        fn(workspace=Tensor((1 << 24,), U8, 1))
    with pytest.raises(ValueError, match="workspace is on cuda:1"):
        K.kmoe_device_error(Tensor((4096,), U8, 1))
    assert not gpu.made and not gpu.lib.launched and not gpu.scratch
