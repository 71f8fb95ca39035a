"""Which kernel a 16-bit product of few rows takes, without a GPU: sizes whose times with either kernel are far apart."""
import os

import pytest

from linear16_sizes import form
from quantized_gemm_quantize_amd import binding
from test_block_abi_cpu import ALIGN, NULL, P, SHAPE, caller

ROWS = ("rows",)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("libw8a8.so not built")
    return binding.load()


# rows, channels, inner: few workgroups of 16 channels and a long inner axis (times of the streaming kernel / of tiles shared
# along the inner axis, us), and many channels of a short one
LONG = [(1, 8, 65536), (1, 64, 16384), (1, 256, 65536), (8, 64, 16384), (8, 1024, 16384), (16, 64, 16384), (16, 256, 9216),
        (16, 8, 1 << 20)]     # 46 / 9, 14 / 7, 50 / 14, 15 / 8, 16 / 12, 18 / 9, 13 / 8, 1361 / 51
WIDE = [(1, 65536, 64), (16, 32000, 64), (16, 65536, 256)]            # 13 / 5.6, 7.6 / 4.1, 16 / 11
STREAM = [(1, 8, 4096), (1, 64, 4096), (16, 64, 4096), (16, 4096, 4096), (1, 4096, 11008), (16, 4096, 8192), (1, 11008, 4096),
          (16, 11008, 4096), (1, 32000, 4096), (16, 32000, 4096), (1, 2048, 8192)]


def test_up_to_16_rows(lib):
    for size in STREAM:
        assert form(lib, *size) == ROWS and lib.w16a16_linear_workspace(*size) == 0, size
    for size in LONG:
        assert form(lib, *size) != ROWS and lib.w16a16_linear_workspace(*size) > 0, size
    for size in WIDE:
        assert form(lib, *size) != ROWS, size
    # none at these widths, which the binding relies on
    for m in (1, 5, 16):
        for n, k in [(n, k) for n in (8, 64, 1000, 4096) for k in (8, 64, 1000, 8192)] + [
                (n, k) for n in (4104, 11008, 1 << 20) for k in (1024, 4096, 8192)]:
            assert form(lib, m, n, k) == ROWS and lib.w16a16_linear_workspace(m, n, k) == 0, (m, n, k)


@pytest.mark.parametrize("M,N,K", LONG)
def test_a_workspace_may_be_left_out_up_to_16_rows(lib, M, N, K):
    """Such a call is valid, and goes as far as any other (here: to the output that is missing)."""
    base = dict(x=P, ldx=K, M=M, w=P, N=N, K=K, dt=0, bias=P, act=1, residual=P, ldr=N, pre=P, out=0, work=0, size=0, stream=None)
    c = caller(lib.w16a16_linear, base)
    need = lib.w16a16_linear_workspace(M, N, K)
    for size in (0, 16, need - 1):
        assert c(size=size) == NULL and c(size=size, work=P) == NULL
    assert c(size=-1) == SHAPE and c(size=need, out=P) == NULL      # a size without an address
    assert c(size=need, work=P + 8, out=P) == ALIGN and c(size=16, work=P + 8, out=P) == ALIGN


# weights that tiles read no faster than memory gives them, a part of a round at a time (streaming kernel / tiles, us): 16.8 /
# 20.1, 17.5 / 20.3, 18.0 / 20.5, 39.5 / 45.8, 43.7 / 46.7
FROM_MEMORY = [(17, 4096, 8192), (24, 4096, 8192), (32, 4096, 8192), (17, 8192, 11008), (24, 8192, 11008)]


def test_17_to_64_rows(lib):
    for size in [*FROM_MEMORY, (24, 4096, 4096), (64, 1024, 1024), (64, 4096, 1024), (24, 1024, 2048)]:
        assert form(lib, *size) == ROWS and lib.w16a16_linear_workspace(*size) == 0, size
    for size in [(64, 4096, 8192), (64, 4096, 11008), (64, 8192, 2048), (64, 11008, 4096), (24, 256, 8192), (24, 16384, 8192)]:
        assert form(lib, *size) != ROWS, size
