"""Sizes of the dense int8 products whose launch would hold 2^32 threads or more are refused before any launch, without
a GPU (pointers here are never dereferenced)."""
import os

import pytest

from quantized_gemm_quantize_amd import binding
from test_block_abi_cpu import NULL, P, SHAPE, caller


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("libw8a8.so not built")
    return binding.load()


def entries(lib):
    operands = dict(xq=P, xs=P, M=1, wq=P, ws=P, N=32, K=16)
    yield caller(lib.w8a8_gemm, {**operands, "out": 0, "dtype": 0, "stream": None})
    yield caller(lib.w8a8_gemm_addmm, {**operands, "bias": P, "alpha": 1.0, "beta": 1.0, "out": 0, "stream": None})
    yield caller(lib.w8a8_gemm_act, {**operands, "bias": P, "act": 1, "residual": 0, "ldr": 0, "out": 0, "stream": None})


def test_channels(lib):
    """A workgroup of up to 512 threads (1024 past K = 4096) for 16 channels, up to 64 rows; larger tiles above."""
    for call in entries(lib):
        for m in (1, 16, 17, 64):
            for k in (16, 2064, 4096):
                assert call(M=m, N=2 ** 27 - 16, K=k) == NULL      # the missing output, further on
                for n in (2 ** 27, 2 ** 28 + 16, 2 ** 30 - 16):
                    assert call(M=m, N=n, K=k) == SHAPE, (m, n, k)
            assert call(M=m, N=2 ** 26 - 16, K=4112) == NULL and call(M=m, N=2 ** 26, K=4112) == SHAPE
        assert call(M=65, N=2 ** 27, K=16) == NULL
