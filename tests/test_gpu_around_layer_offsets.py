"""Elements past 2^31 of every operand and output of the operators around a layer: rows that lie far apart, bit for bit
as their contiguous copies, and whole tensors of more than 2^31 elements, their last rows and channels checked."""
import numpy as np
import pytest
import torch

import block_reference as ref
from quantized_gemm_quantize_amd import binding as b
from test_gpu_linear16_forms import close, product

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16
FAR = 2 ** 31


def generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=BF16):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def far(t):
    """The same rows, the last of them 2^31 elements and more behind the first."""
    m, n = t.shape
    ld = -(-FAR // (m - 1) // 8) * 8 + 8
    rows = torch.as_strided(torch.empty((m - 1) * ld + n, dtype=t.dtype, device=t.device), (m, n), (ld, 1))
    assert ld >= n and (m - 1) * ld > FAR
    return rows.copy_(t)


# the streaming kernel of one and of four groups of rows, tiles of 64 x 64 of both kinds, parts of them, and large ones
@pytest.mark.parametrize("M,N,K", [(5, 72, 136), (16, 64, 16384), (60, 136, 264), (72, 72, 136), (72, 8, 1736), (257, 1040, 1312),
                                   (2200, 1360, 216), (2984, 5880, 2144)])
def test_far_rows_forward(M, N, K):
    g = generator(K)
    x, w, residual, bias = randn(g, M, K), randn(g, N, K), randn(g, M, N), randn(g, N, dtype=torch.float32)
    want = b.w16a16_linear(x, w, bias=bias, activation="silu", residual=residual, pre=True)
    got = b.w16a16_linear(far(x), w, bias=bias, activation="silu", residual=far(residual), pre=True)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("M,N,K", [(5, 72, 136), (60, 136, 264), (300, 520, 328), (600, 72, 136), (3428, 512, 4688), (4960, 4824, 280)])
@pytest.mark.parametrize("a", ["none", "gelu"])
def test_far_rows_gradients(M, N, K, a):
    """Both gradients in one launch and each by itself, with the pass that makes d_pre and the sums of columns."""
    g = generator(N)
    d, x, w, pre = randn(g, M, N), randn(g, M, K), randn(g, N, K), randn(g, M, N) if a != "none" else None
    d_far, x_far = far(d), far(x)
    for kw in (dict(), dict(d_w=False), dict(d_x=False)):
        want = b.w16a16_linear_backward(d, x, w, pre=pre, activation=a, **kw)
        got = b.w16a16_linear_backward(d_far, x_far, w, pre=pre, activation=a, **kw)
        assert all(p is q is None or torch.equal(p, q) for p, q in zip(got, want))


# the streaming kernels, 64 x 64 tiles of both kinds, and the larger ones
@pytest.mark.parametrize("M,N,K", [(5, 272, 512), (16, 272, 4096), (40, 272, 512), (33, 16400, 64), (72, 272, 512), (72, 272, 4112),
                                   (1100, 3008, 272), (4100, 2064, 400), (8200, 8208, 272)])
def test_far_residual_of_the_int8_product(M, N, K):
    g = generator(M)
    xq, wq = (torch.randint(-127, 128, s, generator=g, dtype=torch.int8, device=DEV) for s in ((M, K), (N, K)))
    sx, sw = (torch.rand(n, generator=g, device=DEV) * 0.01 for n in (M, N))
    residual = randn(g, M, N)
    want = b.w8a8_gemm_act(xq, sx, wq, sw, activation="gelu", residual=residual)
    assert torch.equal(b.w8a8_gemm_act(xq, sx, wq, sw, activation="gelu", residual=far(residual)), want)


LONG, OTHER = 65608, 32784      # their product is past 2^31


def test_outputs_past_2_31():
    """out, pre, residual and, of the gradients, d_out, pre and d_pre; sums over the many rows and channels."""
    M, N, K = LONG, OTHER, 8
    g = generator(1)
    x, w, bias = randn(g, M, K), randn(g, N, K), randn(g, N, dtype=torch.float32)
    residual = randn(g, M, N)
    out, pre = b.w16a16_linear(x, w, bias=bias, activation="gelu", residual=residual, pre=True)
    for rows in (slice(0, 300), slice(M // 2, M // 2 + 300), slice(M - 300, M)):      # (one MFMA sums K, in any kernel)
        want = b.w16a16_linear(x[rows], w, bias=bias, activation="gelu", residual=residual[rows], pre=True)
        assert torch.equal(out[rows], want[0]) and torch.equal(pre[rows], want[1])
    del out
    d = residual
    d_x, d_w, d_bias, d_pre = b.w16a16_linear_backward(d, x, w, pre=pre, activation="gelu")
    for rows in (slice(0, 70), slice(M - 70, M)):
        want = b.w16a16_linear_backward(d[rows], x[rows], w, pre=pre[rows], activation="gelu", d_x=False, d_w=False)[3]
        assert torch.equal(d_pre[rows], want)
        close(d_x[rows], *product(d_pre[rows], w.t()), "bf16", "d_x")
    last = d_pre[:, N - 64:]
    close(d_w[N - 64:], *product(last.t(), x.t()), "bf16", "d_w")
    # d_bias is of the unrounded values: half a step of each off the stored ones, and at most 8 additions a row group
    # of 32 rows, 256 groups and 16 slices beside each other
    size = last.double().abs().sum(dim=0)
    limit = size * (ref.HALF["bf16"] * 1.01 + (M / 256 + 64) * ref.U)
    assert ((d_bias[N - 64:].double() - last.double().sum(dim=0)).abs() <= limit).all()


def test_weights_past_2_31():
    """w of the forward product and of d_x, and d_w."""
    M, N, K = 8, LONG, OTHER
    g = generator(2)
    x, w = randn(g, M, K), randn(g, N, K)
    out = b.w16a16_linear(x, w)
    for channels in (slice(0, 64), slice(N - 64, N)):
        close(out[:, channels], *product(x, w[channels]), "bf16", "out")
    d = randn(g, M, N)
    d_x, d_w, _, _ = b.w16a16_linear_backward(d, x, w, d_bias=False)
    for columns in (slice(0, 64), slice(K - 64, K)):
        close(d_x[:, columns], *product(d, w[:, columns].t()), "bf16", "d_x")
    for channels in (slice(0, 64), slice(N - 64, N)):
        close(d_w[channels], *product(d[:, channels].t(), x.t()), "bf16", "d_w")


def test_rows_past_2_31():
    """x of the forward product and of d_w, and d_x."""
    M, N, K = LONG, 8, OTHER
    g = generator(3)
    x, w = randn(g, M, K), randn(g, N, K)
    out = b.w16a16_linear(x, w)
    for rows in (slice(0, 64), slice(M - 64, M)):
        close(out[rows], *product(x[rows], w), "bf16", "out")
    d = randn(g, M, N)
    d_x, d_w, _, _ = b.w16a16_linear_backward(d, x, w, d_bias=False)
    for rows in (slice(0, 64), slice(M - 64, M)):
        close(d_x[rows], *product(d[rows], w.t()), "bf16", "d_x")
    for columns in (slice(0, 64), slice(K - 64, K)):
        close(d_w[:, columns], *product(d.t(), x[:, columns].t()), "bf16", "d_w")


def test_int8_outputs_past_2_31():
    M, N, K = LONG, OTHER, 64
    g = generator(4)
    xq, wq = (torch.randint(-127, 128, s, generator=g, dtype=torch.int8, device=DEV) for s in ((M, K), (N, K)))
    sx, sw = (torch.rand(n, generator=g, device=DEV) * 0.01 for n in (M, N))
    residual = randn(g, M, N)
    out = b.w8a8_gemm_act(xq, sx, wq, sw, activation="silu", residual=residual)
    for rows in (slice(0, 300), slice(M // 2, M // 2 + 300), slice(M - 300, M)):
        want = b.w8a8_gemm_act(xq[rows], sx[rows].clone(), wq, sw, activation="silu", residual=residual[rows])
        assert torch.equal(out[rows], want)


T, H = 262152, 8224      # more than 2^31 elements; widths of whole MXFP4 blocks


def test_norms_past_2_31():
    """Rows of the type, int8 and MXFP4; a row's values do not depend on how many rows there are (above 512)."""
    g = generator(5)
    r, y = randn(g, T, H), randn(g, T, H)
    weight, gate = randn(g, H, dtype=torch.float32), randn(g, H, dtype=torch.float32)
    kw = dict(y=y, post_norm=True, gate=gate, scale=0.5)
    ends = (slice(0, 600), slice(T - 600, T))
    for f in (b.block_norm, b.block_norm_w8a8, b.block_norm_mxfp4):
        got = f(r, weight, **kw)
        for rows in ends:
            want = f(r[rows], weight, **{**kw, "y": y[rows]})
            for p, q in zip(got, want):
                if f is b.block_norm_mxfp4 and p.dim() == 3:      # scales [blocks of 256, rows, 8]
                    assert torch.equal(p[:, rows], q)
                else:
                    assert torch.equal(p[rows], q)
        del got


def test_norm_gradients_past_2_31():
    g = generator(6)
    r, y, d = (randn(g, T, H) for _ in range(3))
    weight, gate = randn(g, H, dtype=torch.float32), randn(g, T, H)
    d_r, d_weight, d_y, _, d_gate = b.block_norm_backward(d, r, weight, d_residual=y, y=y, gate=gate)
    for rows in (slice(0, 600), slice(T - 600, T)):
        want = b.block_norm_backward(d[rows], r[rows], weight, d_residual=y[rows], y=y[rows], gate=gate[rows])
        assert torch.equal(d_r[rows], want[0]) and torch.equal(d_y[rows], want[2]) and torch.equal(d_gate[rows], want[4])
    # d_weight of the last columns: 256 workgroups' partial sums of T / 256 rows each, joined by 32 and 8 additions
    total, size = (torch.zeros(64, dtype=torch.float64, device=DEV) for _ in range(2))
    for at in range(0, T, 1 << 15):
        rows = slice(at, min(at + (1 << 15), T))
        s = (r[rows].float().square().sum(dim=1, dtype=torch.float64) / H + 1e-6).rsqrt()
        term = d[rows, H - 64:].double() * r[rows, H - 64:].double() * s[:, None]
        total += term.sum(dim=0)
        size += term.abs().sum(dim=0)
    limit = size * (T / 256 + 64 + 40) * ref.U
    assert ((d_weight[H - 64:].double() - total).abs() <= limit).all()
    assert np.isfinite(d_weight.cpu().numpy()).all()
