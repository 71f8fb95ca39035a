"""What the binding allocates lives until the library has been called, without a GPU: the library is
a stub that looks up each buffer it is given."""
import contextlib
import weakref

import pytest
import torch

from quantized_gemm_quantize_amd import binding as b


class Gpu(torch.Tensor):
    """A CPU tensor that passes for a GPU tensor."""
    __torch_function__ = torch._C._disabled_torch_function_impl
    is_cuda = True
    log = None

    def get_device(self):
        return 0

    def record_stream(self, stream):
        Gpu.log.append(("record_stream", stream))


def gpu(*shape, dtype):
    return torch.zeros(shape, dtype=dtype).as_subclass(Gpu)


class Log(list):
    allocations = None


class Allocations:
    """Stands for torch.empty: remembers what it made, by address, without keeping it alive, and the
    stream that was current then."""

    def __init__(self):
        self.made, self.current, self.streams = {}, None, []

    def __call__(self, *shape, dtype=None, device=None):
        shape = shape[0] if shape and isinstance(shape[0], (tuple, list)) else shape
        t = torch.ones(shape, dtype=dtype).as_subclass(Gpu)
        self.made[t.data_ptr()] = weakref.ref(t)
        self.streams.append(self.current)
        return t


class Library:
    """Every entry point succeeds; buffers that torch.empty made have to be alive when it is called."""

    def __init__(self, allocations, log):
        self.allocations, self.log = allocations, log

    def __getattr__(self, name):
        def entry(*args):
            if name.endswith("_workspace"):
                return 4096
            made = [a for a in args if a in self.allocations.made]
            self.log.append((name, len(made), all(self.allocations.made[a]() is not None for a in made)))
            return b.W8A8_OK
        return entry


@pytest.fixture
def calls(monkeypatch):
    log, allocations = Log(), Allocations()
    Gpu.log = log
    monkeypatch.setattr(torch, "empty", allocations)
    monkeypatch.setattr(b, "load", lambda: Library(allocations, log))
    monkeypatch.setattr(b, "_stream_of", lambda t, stream: 0)
    monkeypatch.setattr(b, "_stream_handle", lambda stream: 0)

    @contextlib.contextmanager
    def current(stream):
        allocations.current = stream
        yield
        allocations.current = None

    monkeypatch.setattr(torch.cuda, "stream", current)
    log.allocations = allocations
    return log


def linear(**kw):
    b.mxfp4_linear(gpu(40, 64, dtype=torch.bfloat16), gpu(32, 32, dtype=torch.uint8), gpu(1, 32, 8, dtype=torch.uint8), **kw)


def sort(**kw):
    b.moe_sort(gpu(3000, 2, dtype=torch.int64), 8, **kw)


def layer(**kw):
    b.mxfp4_moe(gpu(40, 64, dtype=torch.bfloat16), gpu(40, 2, dtype=torch.int64), gpu(40, 2, dtype=torch.float32),
                gpu(3, 64, 32, dtype=torch.uint8), gpu(3, 1, 64, 8, dtype=torch.uint8),
                gpu(3, 64, 16, dtype=torch.uint8), gpu(3, 1, 64, 8, dtype=torch.uint8), **kw)


@pytest.mark.parametrize("call,name,buffers", [(linear, "mxfp4_linear", 2), (sort, "moe_sort", 4), (layer, "mxfp4_moe", 2)])
def test_workspace_lives_through_the_call(calls, call, name, buffers):
    """Outputs and the workspace, all of them made by the binding, are alive during the call."""
    call()
    assert [c for c in calls if c[0] == name] == [(name, buffers, True)]


U8, I8, I32, F32, BF16 = torch.uint8, torch.int8, torch.int32, torch.float32, torch.bfloat16


def products():
    """Every entry point that makes its outputs, and the number of tensors that it makes."""
    x, xq, xs, wq, ws = (gpu(8, 256, dtype=BF16), gpu(8, 256, dtype=I8), gpu(8, dtype=F32), gpu(64, 256, dtype=I8),
                         gpu(64, dtype=F32))
    values, meta = gpu(2, 64, 64, dtype=I8), gpu(2, 64, 4, dtype=I32)
    bsr = gpu(2, dtype=I32), gpu(1, dtype=I32), gpu(1, 64, 64, dtype=I8)
    w4 = gpu(64, 128, dtype=U8), gpu(64, 4, dtype=BF16), gpu(64, 4, dtype=BF16)
    mx, mw = (gpu(8, 128, dtype=U8), gpu(1, 8, 8, dtype=U8)), (gpu(64, 128, dtype=U8), gpu(1, 64, 8, dtype=U8))
    ew = gpu(3, 64, 128, dtype=U8), gpu(3, 1, 64, 8, dtype=U8)
    pos, w, rows, offsets = gpu(4, 2, dtype=I32), gpu(4, 2, dtype=F32), gpu(8, 256, dtype=BF16), gpu(4, dtype=I32)
    yield b.w8a8_quantize_rows, (x,), 2
    yield b.w8a8_quantize_rows_f32, (gpu(8, 256, dtype=F32),), 2
    yield b.w8a8_gemm, (xq, xs, wq, ws), 1
    yield b.w8a8_gemm_addmm, (xq, xs, wq, ws), 1
    yield b.w8a8_compress24, (wq,), 2
    yield b.w8a8_sparse24_gemm, (xq, xs, values, meta, ws), 1
    yield b.w4a16_dequant, w4, 1
    yield b.w4a16_gemm, (x, *w4), 1
    yield b.w8a8_bsr_gemm, (xq, xs, *bsr, ws), 1
    yield b.w8a8_bsr_gemm_addmm, (xq, xs, *bsr, ws), 1
    yield b.w8a8_fused_linear, (x, wq, ws), 1
    yield b.w8a8_linear, (x, wq, ws), 3
    yield b.mxfp4_quantize_rows, (x,), 2
    yield b.mxfp4_dequantize_rows, mx, 1
    yield b.mxfp4_gemm, (*mx, *mw), 1
    yield b.mxfp4_linear, (x, *mw), 2
    yield b.moe_sort, (gpu(4, 2, dtype=torch.int64), 3), 4
    yield b.moe_gather, (gpu(4, 256, dtype=BF16), pos), 1
    yield b.moe_gather_backward, (rows, pos), 1
    yield b.moe_combine, (rows, pos, w), 1
    yield b.moe_combine_backward, (gpu(4, 256, dtype=BF16), rows, pos, w), 2
    yield b.mxfp4_expert_gemm, (*mx, offsets, *ew), 1
    yield b.mxfp4_expert_swiglu, (*mx, offsets, *ew), 2
    yield b.mxfp4_moe, (gpu(4, 64, dtype=BF16), gpu(4, 2, dtype=torch.int64), w, gpu(3, 64, 32, dtype=U8),
                        gpu(3, 1, 64, 8, dtype=U8), gpu(3, 64, 16, dtype=U8), gpu(3, 1, 64, 8, dtype=U8)), 2


@pytest.mark.parametrize("index", range(len(list(products()))))
def test_new_tensors_belong_to_the_stream_that_writes_them(calls, index):
    """With stream=, outputs and workspaces come from that stream's pool: memory freed on the current
    stream with work still queued there is not written by another stream, and what is dropped early is
    reused in that stream's order. Without, they come from the current stream's."""
    call, args, tensors = list(products())[index]
    call(*args)
    assert calls.allocations.streams == [None] * tensors, call.__name__
    calls.allocations.streams.clear()
    side = object()
    call(*args, stream=side)
    assert calls.allocations.streams == [side] * tensors, call.__name__
