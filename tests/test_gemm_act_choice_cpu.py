"""Which kernel the int8 product with its epilogue takes, without a GPU: sizes whose times with the kernels are far
apart."""
import ctypes
import os

import pytest

from quantized_gemm_quantize_amd import binding

STREAMING, OWN_STAGES, TILES_64, TILES = range(4)


@pytest.fixture(scope="module")
def form():
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("libw8a8.so not built")
    f = binding.load().w8a8_act_debug_form
    f.argtypes = [ctypes.c_int64] * 3
    return f


def test_17_to_64_rows_of_many_channels(form):
    """Streaming / 64 x 64 tiles, us: 64 x 32000 x 11008 257 / 87, 64 x 16640 x 8208 130 / 70, 64 x 32000 x 1024 40 / 12,
    32 x 32000 x 8192 107 / 53, 17 x 32000 x 2048 25 / 18."""
    for m in (17, 32, 33, 64):
        for n in (16400, 16640, 32000, 1 << 20):
            for k in (64, 1024, 2048, 8192, 8208, 11008):
                assert form(m, n, k) == TILES_64, (m, n, k)
    for n in (16400, 32000, 1 << 20):
        assert form(16, n, 8208) == STREAMING


def test_33_to_64_rows(form):
    """Wavefronts with stages of their own / 64 x 64 tiles, us: 64 x 4096 x 2048 8.0 / 10.2, 48 x 2048 x 3584 9.4 / 14.3,
    33 x 16384 x 2048 10.8 / 14.8."""
    for m in (33, 48, 64):
        for n in (2048, 4096, 16384):
            for k in (2048, 3088, 4080, 4096, 11008):
                assert form(m, n, k) == OWN_STAGES, (m, n, k)
        for n in (64, 1024, 2032):
            assert form(m, n, 2048) == STREAMING
        for n in (64, 4096, 16384):
            assert form(m, n, 1024) == STREAMING


def test_other_sizes_stay(form):
    for size, want in {(1, 4096, 4096): STREAMING, (16, 11008, 4096): STREAMING, (24, 4096, 4096): STREAMING,
                       (24, 11008, 4096): OWN_STAGES, (64, 1344, 5840): OWN_STAGES, (128, 4096, 11008): OWN_STAGES,
                       (256, 2176, 8064): OWN_STAGES, (633, 288, 272): TILES_64, (256, 11008, 4096): TILES_64,
                       (65, 4096, 2048): TILES_64, (400, 4096, 4096): TILES_64, (2048, 4096, 4096): TILES,
                       (8200, 8208, 256): TILES, (1000, 4096, 4096): TILES}.items():
        assert form(*size) == want, size
