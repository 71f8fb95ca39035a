"""What the binding allocates lives until the library has been called, without a GPU: the library is
a stub that looks up each buffer it is given."""
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


class Allocations:
    """Stands for torch.empty: remembers what it made, by address, without keeping it alive."""

    def __init__(self):
        self.made = {}

    def __call__(self, *shape, dtype=None, device=None):
        shape = shape[0] if shape and isinstance(shape[0], (tuple, list)) else shape
        t = torch.ones(shape, dtype=dtype).as_subclass(Gpu)
        self.made[t.data_ptr()] = weakref.ref(t)
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
    log, allocations = [], Allocations()
    Gpu.log = log
    monkeypatch.setattr(torch, "empty", allocations)
    monkeypatch.setattr(b, "load", lambda: Library(allocations, log))
    monkeypatch.setattr(b, "_stream_of", lambda t, stream: 0)
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
