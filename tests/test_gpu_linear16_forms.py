"""16-bit products through every compiled variant of their kernels, forward and both gradients' operand layouts,
against 64 bits."""
import pytest
import torch

import block_reference as ref
from linear16_sizes import PAIRS, ROWS, TILED
from quantized_gemm_quantize_amd import binding as b

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def rows(g, m, n, dtype, size=1.0, extra=8):
    """Rows of a stride of n + extra, NaN between them."""
    t = torch.full((m, n + extra), float("nan"), dtype=TYPES[dtype], device=DEV)[:, :n]
    t.copy_(torch.randn((m, n), generator=g, device=DEV) * size)
    return t


def product(a, w):
    """(a w^T, its bound) in 64 bits: the bound of the reference module's product."""
    steps = a.shape[1] / 8 + 16
    a, w = a.double().contiguous(), w.double()
    return a @ w.t().contiguous(), a.abs() @ w.abs().t().contiguous() * (steps * 2.0 ** -23)


def close(got, want, bound, dtype, what):
    limit = bound + (want.abs() + bound) * ref.HALF[dtype] + ref.TINY[dtype]
    off = (got.double() - want).abs() / limit
    assert bool((off <= 1).all()), f"{what}: the worst by {off.nan_to_num(9e9).max().item()} of its bound"


@pytest.mark.parametrize("M,N,K", ROWS + TILED)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_forward(dtype, M, N, K):
    """relu (whose value is exact), with everything that an epilogue has, in place of the residual."""
    g = torch.Generator(device=DEV).manual_seed(M + N + K)
    x, w = rows(g, M, K, dtype), rows(g, N, K, dtype, K ** -0.5, extra=0)
    bias = torch.randn(N, generator=g, device=DEV)
    buffer = torch.full((M + 3, N), 5.0, dtype=TYPES[dtype], device=DEV)
    buffer[:M] = torch.randn((M, N), generator=g, device=DEV)
    residual = buffer[:M].clone()
    out, pre = b.w16a16_linear(x, w, bias=bias, activation="relu", residual=buffer[:M], pre=True, out=buffer[:M])
    want, e = product(x, w)
    want = want + bias.double()
    e = e + ref.U * want.abs()
    close(pre, want, e, dtype, "pre")
    want = want.clamp(min=0) + residual.double()
    close(out, want, e + ref.U * want.abs(), dtype, "out")
    assert (buffer[M:] == 5).all()


@pytest.mark.parametrize("M,N,K", TILED)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gradients(dtype, M, N, K):
    """A product of the size as d_x (its second operand runs along the inner axis) and as d_w (both do)."""
    g = torch.Generator(device=DEV).manual_seed(M + 2 * N + K)
    d, x, w = rows(g, M, K, dtype), rows(g, M, N, dtype), rows(g, K, N, dtype, K ** -0.5, extra=0)
    got = b.w16a16_linear_backward(d, x, w, d_w=False, d_bias=False)[0]
    close(got, *product(d, w.t()), dtype, "d_x")
    d, x = rows(g, K, M, dtype, K ** -0.5), rows(g, K, N, dtype)
    got = b.w16a16_linear_backward(d, x, torch.empty((M, N), dtype=TYPES[dtype], device=DEV), d_x=False, d_bias=False)[1]
    close(got, *product(d.t(), x.t()), dtype, "d_w")
    again = b.w16a16_linear_backward(d, x, torch.empty((M, N), dtype=TYPES[dtype], device=DEV), d_x=False, d_bias=False)[1]
    assert torch.equal(got, again)


@pytest.mark.parametrize("M,N,K", PAIRS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_both_gradients(dtype, M, N, K):
    """In one launch, against 64 bits and against one by one."""
    g = torch.Generator(device=DEV).manual_seed(M + 3 * N + K)
    d, x, w = rows(g, M, N, dtype, N ** -0.5), rows(g, M, K, dtype), rows(g, N, K, dtype, extra=0)
    need = b.w16a16_linear_backward_workspace(M, N, K)
    work = torch.full((need + 4096,), 77, dtype=torch.uint8, device=DEV)
    d_x, d_w, d_bias, _ = b.w16a16_linear_backward(d, x, w, workspace=work[:need])
    assert (work[need:] == 77).all()
    close(d_x, *product(d, w.t()), dtype, "d_x")
    close(d_w, *product(d.t(), x.t()), dtype, "d_w")
    again = b.w16a16_linear_backward(d, x, w)
    assert torch.equal(d_x, again[0]) and torch.equal(d_w, again[1]) and torch.equal(d_bias, again[2])
