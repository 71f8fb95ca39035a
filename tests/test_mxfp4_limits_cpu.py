"""The largest sizes of the MXFP4 and expert entry points, without a GPU: a launch holds fewer than 2^32
threads, and sizes past that get the status of a shape, before any pointer is looked at."""
import os

import pytest

from quantized_gemm_quantize_amd import binding

NULL, SHAPE = -1, -2
P = 0x10000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("libw8a8.so not built")
    return binding.load()


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("k", [32, 256, 512, 4096])
def test_rows(lib, dtype, k):
    """32 threads per 256 elements, in workgroups of 256."""
    most = (2 ** 27 - 8) // (-(-k // 256))
    assert lib.mxfp4_quantize_rows(0, k, most, k, dtype, P, P, None) == NULL
    assert lib.mxfp4_quantize_rows(0, k, most + 1, k, dtype, P, P, None) == SHAPE
    assert lib.mxfp4_dequantize_rows(0, P, most, k, dtype, P, None) == NULL
    assert lib.mxfp4_dequantize_rows(0, P, most + 1, k, dtype, P, None) == SHAPE


# rows, experts; rows of a workgroup, its channels, its threads (the kernels for a few rows per
# expert, and the smallest tile)
GROUPED = [(6144, 512, 16, 64, 128), (12288, 512, 32, 64, 128), (12289, 512, 64, 128, 256),
           (512, 512, 16, 64, 128)]


@pytest.mark.parametrize("S,E,rows,channels,threads", GROUPED)
def test_expert_products(lib, S, E, rows, channels, threads):
    tiles = min(S, S // rows + E + 1)
    most = (2 ** 32 - 1) // (tiles * threads) * channels      # channels that still fit
    assert most * S <= 2 ** 36 and most < 2 ** 27
    for n, status in ((most, NULL), (most + channels, SHAPE)):
        assert lib.mxfp4_expert_gemm(0, P, S, None, S, P, E, P, P, n, 32, 0, P, None) == status


def test_layer(lib):
    """Bounds of the layer's parts leave its launches within a grid: the products of few rows for each
    of 512 experts at the widest hidden rows, and the sort's, which quantizes the tokens too (32 steps of 256
    elements, or 4096 slots, per workgroup of 1024 threads), at the most tokens of any width."""
    assert 897 * (2 * binding.MXFP4_MAX_K // 64) * 128 < 2 ** 32
    assert lib.mxfp4_moe_workspace(6144, 1, 512, 32, binding.MXFP4_MAX_K, 0) > 0
    for h in (32, 288, 544, 1056, 4096, 65536):
        t = min((2 ** 32 - 1) // (h // 2), 2 ** 24 - 1, (2 ** 27 - 8) // -(-h // 256))
        assert lib.mxfp4_moe_workspace(t, 1, 8, h, 32, 0) > 0
        assert (-(-t * -(-h // 256) // 32) + -(-t // 4096)) * 1024 < 2 ** 32
    assert lib.mxfp4_moe_workspace(2 ** 21, 1, 8, 4096, 32, 0) == 0
