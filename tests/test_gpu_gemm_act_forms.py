"""The int8 product with its epilogue through every kernel that carries it, whole and ragged stages, against 64 bits and
against the plain int8 product, bit for bit where they compute the same."""
import os

import pytest
import torch

import block_reference as ref
from gpu_layer import library
from quantized_gemm_quantize_amd import binding as b
from quantized_gemm_quantize_amd.build import POISON_LIB

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
# 64 x 64 tiles (a round of them, and 33 to 64 rows of many channels; wavefronts with stages of their own), 128 x 64, 256 x 128 at one and at two workgroups
# per CU, 256 x 256, the streaming kernels
SIZES = [(64, 2064, 2064), (50, 2048, 2048), (300, 1040, 4112), (256, 2048, 4096), (20, 8208, 4096), (65, 16, 8208), (65, 144, 528), (300, 1040, 1024), (40, 2064, 400), (64, 2048, 1024), (33, 11008, 4096), (1100, 3008, 272), (1000, 4096, 256),
         (4100, 2064, 400), (4096, 2048, 1024), (8200, 8208, 272), (8200, 8208, 256), (8200, 8208, 1040), (8192, 8192, 1152),
         (1, 4096, 4096), (16, 272, 8192), (24, 2064, 1040), (48, 1040, 1024), (64, 4096, 8208)]


def case(M, N, K):
    g = torch.Generator(device=DEV).manual_seed(M + N + K)
    xq, wq = (torch.randint(-127, 128, s, generator=g, dtype=torch.int8, device=DEV) for s in ((M, K), (N, K)))
    sx, sw = (2.0 ** (torch.rand(n, generator=g, device=DEV) * 4 - 9) for n in (M, N))
    sw = sw * K ** -0.5
    bias = torch.randn(N, generator=g, device=DEV)
    residual = torch.randn((M, N), generator=g, device=DEV).to(torch.bfloat16)
    return xq, sx, wq, sw, bias, residual


@pytest.mark.parametrize("M,N,K", SIZES)
def test_forms(M, N, K):
    xq, sx, wq, sw, bias, residual = case(M, N, K)
    assert torch.equal(b.w8a8_gemm_act(xq, sx, wq, sw), b.w8a8_gemm(xq, sx, wq, sw))
    buffer = torch.full((M + 3, N), 5.0, dtype=torch.bfloat16, device=DEV)
    buffer[:M] = residual
    out = b.w8a8_gemm_act(xq, sx, wq, sw, bias=bias, activation="relu", residual=buffer[:M], out=buffer[:M])
    assert (buffer[M:] == 5).all()
    acc = (xq.double() @ wq.double().t().contiguous()) * sx.double()[:, None] * sw.double()[None, :]
    want = acc + bias.double()
    # two roundings of the scaled sum (the integer's own included: three), one of the bias, one of the residual
    e = 3 * ref.U * acc.abs() + ref.U * want.abs()
    want = want.clamp(min=0) + residual.double()
    e = e + ref.U * want.abs()
    limit = e + (want.abs() + e) * ref.HALF["bf16"] + ref.TINY["bf16"]
    off = ((out.double() - want).abs() / limit).nan_to_num(9e9).max().item()
    assert off <= 1, off


@pytest.mark.parametrize("M,N,K", SIZES)
def test_lds_poisoned(M, N, K):
    xq, sx, wq, sw, bias, residual = case(M, N, K)
    want = b.w8a8_gemm_act(xq, sx, wq, sw, bias=bias, activation="silu", residual=residual)
    torch.cuda.synchronize()
    assert os.path.exists(POISON_LIB)
    with library(POISON_LIB) as poisoned:
        got = poisoned.w8a8_gemm_act(xq, sx, wq, sw, bias=bias, activation="silu", residual=residual)
        torch.cuda.synchronize()
    assert torch.equal(got, want)
