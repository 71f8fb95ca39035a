"""The int8 product with its epilogue for 17 to 64 rows of many channels, and of an inner axis from 2048 on, as the other
sizes are tested: against 64 bits, the plain product and the LDS-poisoned build."""
import pytest

import test_gpu_gemm_act_forms as forms

pytestmark = pytest.mark.gpu
SIZES = [(17, 16400, 64), (24, 50000, 272), (32, 16640, 4096), (40, 20000, 1040), (50, 16640, 4112), (64, 32000, 8208),
         (33, 2048, 2048), (48, 3008, 3088), (64, 16384, 2064), (64, 4096, 4080)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_forms(M, N, K):
    forms.test_forms(M, N, K)


@pytest.mark.parametrize("M,N,K", SIZES)
def test_lds_poisoned(M, N, K):
    forms.test_lds_poisoned(M, N, K)
