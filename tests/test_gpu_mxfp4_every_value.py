"""MXFP4 quantization of every 16-bit value at every scale it can be rounded under."""
import numpy as np
import pytest
import torch

import mx_reference as ref
from quantized_gemm_quantize_amd import binding as b
from test_gpu_mxfp4 import DEV, TYPES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_value_under_every_scale(dtype):
    """For every power of two as a block's largest exponent, all values of both signs from that binade
    down to a 32nd of it (smaller ones are 0), in blocks behind the power of two itself: elements, scales
    and the values back are exact."""
    every = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(TYPES[dtype])
    every = every[torch.isfinite(every)]
    mag = every.double().abs()
    low, high = (-133, 127) if dtype == "bf16" else (-24, 15)
    blocks = []
    for e in range(low, high + 1):
        v = every[(mag < 2.0 ** (e + 1)) & (mag >= 2.0 ** (e - 5))]
        v = torch.cat([v, v.new_zeros(-len(v) % 31)]).reshape(-1, 31)
        blocks.append(torch.cat([v.new_full((len(v), 1), 2.0 ** e), v], dim=1))
    x = torch.cat(blocks)
    assert len(x) > 10000
    codes, scales = b.mxfp4_quantize_rows(x.to(DEV))
    q, code = ref.quantize(x.double().numpy())
    c, s = ref.pack(q, code)
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)
    back = b.mxfp4_dequantize_rows(codes, scales, TYPES[dtype])
    assert torch.equal(back.cpu(), torch.from_numpy(ref.values(q, code)).to(TYPES[dtype]))


def test_single_precision_around_every_boundary():
    """fp32 values at, next below and next above every rounding boundary of the grid, and of the scale
    itself, for every exponent with its subnormals."""
    grid = np.array([0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0, 7.9999995], dtype=np.float32)
    rows = []
    for e in range(-149, 125):                                # 8 * 2^e is still finite
        v = np.ldexp(grid.astype(np.float64), e).astype(np.float32)          # the top's own exponent is e + 2
        near = np.concatenate([v, np.nextafter(v, np.float32(0)), np.nextafter(v, np.float32(np.inf))])
        near = near[near.astype(np.float64) < 2.0 ** (e + 3)]
        near = np.concatenate([near, -near])
        near = np.concatenate([near, np.zeros(-len(near) % 31, dtype=np.float32)]).reshape(-1, 31)
        top = np.full((len(near), 1), np.ldexp(np.float32(1), e + 2), dtype=np.float32)
        rows.append(np.concatenate([top, near], axis=1))
    x = np.concatenate(rows)
    codes, scales = b.mxfp4_quantize_rows(torch.from_numpy(x).to(DEV))
    c, s = ref.pack(*ref.quantize(x.astype(np.float64)))
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)
