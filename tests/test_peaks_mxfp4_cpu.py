"""The MXFP4 reference rates of libpeaks.so reject malformed arguments before any HIP call."""
import ctypes
import os

import pytest

from quantized_gemm_quantize_amd.build import PEAKS_LIB


def test_bad_arguments_rejected_on_the_host():
    if not os.path.exists(PEAKS_LIB):
        pytest.skip("libpeaks.so not built")
    lib = ctypes.CDLL(PEAKS_LIB)
    p, i32 = ctypes.c_void_p, ctypes.c_int
    lib.peaks_operand_stream256.argtypes = [p, p, i32, i32, i32, p, p]
    lib.peaks_mfma_mxfp4.argtypes = [i32, i32, p, p, p]
    fake = ctypes.c_void_p(16)   # never dereferenced: every call below fails its checks first
    for m, n, k in ((128, 256, 128), (256, 128, 128), (256, 256, 64), (0, 256, 128), (256, 256, 0), (256, -256, 128)):
        assert lib.peaks_operand_stream256(fake, fake, m, n, k, fake, None) == -1
    assert lib.peaks_operand_stream256(None, fake, 256, 256, 128, fake, None) == -1
    assert lib.peaks_operand_stream256(fake, fake, 256, 256, 128, None, None) == -1
    assert lib.peaks_mfma_mxfp4(0, 1, fake, fake, None) == -1
    assert lib.peaks_mfma_mxfp4(1, 1, None, fake, None) == -1
