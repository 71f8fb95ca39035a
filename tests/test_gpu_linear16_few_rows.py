"""16-bit products of up to 16 rows whose inner axis is shared by tiles, or whose channels are many, with the workspace that
they ask for and without one, against 64 bits."""
import pytest
import torch

import block_reference as ref
from quantized_gemm_quantize_amd import binding as b
from test_gpu_linear16_forms import DEV, TYPES, close, product, rows

pytestmark = pytest.mark.gpu
SIZES = [(1, 8, 65536), (2, 72, 16392), (5, 264, 20488), (9, 1000, 16400), (16, 64, 16384), (16, 256, 9216), (16, 8, 1 << 20),
         (16, 4104, 64), (3, 65536, 64), (16, 32008, 72)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_with_and_without_a_workspace(dtype, M, N, K):
    g = torch.Generator(device=DEV).manual_seed(M + N + K)
    x, w = rows(g, M, K, dtype), rows(g, N, K, dtype, K ** -0.5, extra=0)
    bias = torch.randn(N, generator=g, device=DEV)
    kept = torch.randn((M, N), generator=g, device=DEV).to(TYPES[dtype])
    need = b.w16a16_linear_workspace(M, N, K)
    want, e = product(x, w)
    want = want + bias.double()
    e = e + ref.U * want.abs()
    out_want = want.clamp(min=0) + kept.double()
    e_out = e + ref.U * out_want.abs()
    for size in (None, need, 0, need // 2):
        work = None if size is None else torch.full((size + 256,), 77, dtype=torch.uint8, device=DEV)
        buffer = torch.full((M + 3, N), 5.0, dtype=TYPES[dtype], device=DEV)
        buffer[:M] = kept
        args = dict(bias=bias, activation="relu", residual=buffer[:M], pre=True, out=buffer[:M],
                    workspace=None if work is None else work[:size])
        out, pre = b.w16a16_linear(x, w, **args)
        close(pre, want, e, dtype, f"pre {size}")
        close(out, out_want, e_out, dtype, f"out {size}")
        assert (buffer[M:] == 5).all() and (work is None or (work[size:] == 77).all())
        buffer[:M] = kept
        again, _ = b.w16a16_linear(x, w, **args)
        assert torch.equal(again, out)


def test_captured_without_a_workspace():
    """Both forms of one product in a graph, replayed with eager work between."""
    M, N, K = 16, 64, 16384
    g = torch.Generator(device=DEV).manual_seed(3)
    x, w = rows(g, M, K, "bf16"), rows(g, N, K, "bf16", K ** -0.5, extra=0)
    none = torch.empty(0, dtype=torch.uint8, device=DEV)

    def run():
        return [b.w16a16_linear(x, w, activation="silu"), b.w16a16_linear(x, w, activation="silu", workspace=none)]

    want = run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(4):
        for t in got:
            t.zero_()
        b.w16a16_linear(x, w)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(got, want))
