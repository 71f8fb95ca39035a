"""What the binding allocates for the block norms and the 16-bit products, on which stream, and what it refuses,
without a GPU."""
import types

import pytest
import torch

from quantized_gemm_quantize_amd import binding as b
from test_binding_lifetimes_cpu import Gpu, calls, gpu  # noqa: F401 (calls is a fixture)

I8, F32, BF16, F16 = torch.int8, torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def device(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)


def entries():
    """Every entry point, its arguments, and the number of tensors that it makes."""
    x, w, rows, v = gpu(8, 256, dtype=BF16), gpu(64, 256, dtype=BF16), gpu(8, 64, dtype=BF16), gpu(256, dtype=F32)
    q = gpu(8, 256, dtype=I8), gpu(8, dtype=F32), gpu(64, 256, dtype=I8), gpu(64, dtype=F32)
    yield b.w8a8_gemm_act, q, dict(bias=gpu(64, dtype=F32), residual=rows), 1
    many = gpu(40, 256, dtype=BF16), w
    yield b.w16a16_linear, (x, w), dict(activation="silu"), 1      # up to 16 rows need no workspace
    yield b.w16a16_linear, many, dict(activation="silu"), 2
    yield b.w16a16_linear, many, dict(activation="gelu", pre=True, residual=gpu(40, 64, dtype=BF16)), 3
    yield b.w16a16_linear_backward, (rows, x, w), dict(), 4
    yield b.w16a16_linear_backward, (rows, x, w), dict(pre=rows, activation="relu", d_x=False), 4
    yield b.block_norm, (x,), dict(), 1
    yield b.block_norm, (x, v), dict(y=x, gate=x), 2
    yield b.block_norm_w8a8, (x, v), dict(y=x, post_weight=v), 3
    yield b.block_norm_mxfp4, (x,), dict(y=x, gate=v), 3
    yield b.block_norm_backward, (x, x), dict(), 3
    yield b.block_norm_backward, (x, x, v), dict(y=x, gate=v, post_norm=True), 6


@pytest.mark.parametrize("index", range(len(list(entries()))))
def test_new_tensors(calls, index):  # noqa: F811
    """Outputs and workspaces are alive during the call, and come from the pool of the stream that writes them."""
    f, args, kw, tensors = list(entries())[index]
    f(*args, **kw)
    assert [c for c in calls if c[0] == f.__name__] == [(f.__name__, tensors, True)]
    assert calls.allocations.streams == [None] * tensors
    calls.allocations.streams.clear()
    side = types.SimpleNamespace(cuda_stream=0)
    f(*args, **kw, stream=side)
    assert calls.allocations.streams == [side] * tensors


@pytest.mark.parametrize("index", range(len(list(entries()))))
def test_other_devices_are_refused(calls, index, monkeypatch):  # noqa: F811
    """A launch goes to the current device: tensors of another one, or of two, are refused before it."""
    f, args, kw, _ = list(entries())[index]
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    with pytest.raises(ValueError, match="current device"):
        f(*args, **kw)
    monkeypatch.undo()
    assert not [c for c in calls if c[0] == f.__name__]


class Elsewhere(Gpu):
    def get_device(self):
        return 1


@pytest.mark.parametrize("index", range(len(list(entries()))))
def test_tensors_of_two_devices_are_refused(calls, index):  # noqa: F811
    f, args, kw, _ = list(entries())[index]
    for i in range(1, len(args)):
        moved = [a.as_subclass(Elsewhere) if j == i else a for j, a in enumerate(args)]
        with pytest.raises(ValueError, match="device"):
            f(*moved, **kw)
    for name, t in kw.items():
        if isinstance(t, torch.Tensor):
            with pytest.raises(ValueError, match="device"):
                f(*args, **{**kw, name: t.as_subclass(Elsewhere)})
    assert not [c for c in calls if c[0] == f.__name__]


def test_arguments(calls):  # noqa: F811
    x, w, rows, v = gpu(8, 256, dtype=BF16), gpu(64, 256, dtype=BF16), gpu(8, 64, dtype=BF16), gpu(256, dtype=F32)
    bad = [
        (b.w16a16_linear, (x, w), dict(activation="swish")), (b.w16a16_linear, (x, w), dict(activation=2)),
        (b.w16a16_linear, (gpu(8, 256, dtype=F32), w), {}), (b.w16a16_linear, (gpu(8, 256, dtype=F16), w), {}),
        (b.w16a16_linear, (x, gpu(64, 128, dtype=BF16)), {}), (b.w16a16_linear, (x, w), dict(bias=gpu(65, dtype=F32))),
        (b.w16a16_linear, (x, w), dict(bias=gpu(64, dtype=BF16))), (b.w16a16_linear, (x, w), dict(residual=x)),
        (b.w16a16_linear, (x, w), dict(residual=gpu(8, 64, dtype=F32))),
        (b.w16a16_linear, (x, w), dict(out=gpu(8, 65, dtype=BF16))), (b.w16a16_linear, (x, w), dict(pre=gpu(8, 64, dtype=F16))),
        (b.w16a16_linear, (x, w), dict(workspace=gpu(8, dtype=I8))), (b.w16a16_linear, (None, w), {}),
        (b.w16a16_linear_backward, (None, x, w), {}), (b.w16a16_linear_backward, (x, x, w), {}),
        (b.w16a16_linear_backward, (rows, x, w), dict(activation="gelu")),
        (b.w16a16_linear_backward, (rows, x, w), dict(activation="gelu", pre=x)),
        (b.w16a16_linear_backward, (rows, x, w), dict(d_x=rows)), (b.w16a16_linear_backward, (rows, x, w), dict(d_bias=v)),
        (b.block_norm, (x, gpu(255, dtype=F32)), {}), (b.block_norm, (x, gpu(256, dtype=BF16)), {}),
        (b.block_norm, (x,), dict(gate=v)), (b.block_norm, (x,), dict(post_norm=True)), (b.block_norm, (x,), dict(post_weight=v)),
        (b.block_norm, (x,), dict(new_residual=x)), (b.block_norm, (x,), dict(y=rows)), (b.block_norm, (x,), dict(y=gpu(8, 256, dtype=F16))),
        (b.block_norm, (x,), dict(y=x, gate=gpu(8, 256, dtype=F32))), (b.block_norm, (x,), dict(y=x, gate=gpu(8, dtype=F32))),
        (b.block_norm, (x,), dict(out=gpu(8, 256, dtype=F32))), (b.block_norm, (gpu(8, 256, dtype=torch.float64),), {}),
        (b.block_norm_w8a8, (x,), dict(xq=x)), (b.block_norm_mxfp4, (x,), dict(scales=gpu(2, 8, 8, dtype=torch.uint8))),
        (b.block_norm_backward, (None, x), {}), (b.block_norm_backward, (rows, x), {}),
        (b.block_norm_backward, (x, x), dict(gate=v)), (b.block_norm_backward, (x, x), dict(post_norm=True)),
        (b.block_norm_backward, (x, x), dict(workspace=gpu(16, dtype=I8))),
        (b.w8a8_gemm_act, (gpu(8, 256, dtype=I8), gpu(8, dtype=F32), gpu(64, 256, dtype=I8), gpu(64, dtype=F32)), dict(residual=x)),
        (b.w8a8_gemm_act, (gpu(8, 256, dtype=I8), gpu(9, dtype=F32), gpu(64, 256, dtype=I8), gpu(64, dtype=F32)), {}),
    ]
    for f, args, kw in bad:
        with pytest.raises((ValueError, TypeError)):
            f(*args, **kw)
            pytest.fail(f"{f.__name__} {kw}")
    names = {"w16a16_linear", "w16a16_linear_backward", "block_norm", "block_norm_w8a8", "block_norm_mxfp4",
             "block_norm_backward", "w8a8_gemm_act"}
    assert not [c for c in calls if c[0] in names]
