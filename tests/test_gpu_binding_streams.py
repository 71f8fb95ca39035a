"""Calls on a stream of their own whose outputs and workspaces the binding allocates."""
import pytest
import torch

from quantized_gemm_quantize_amd import binding as b
from test_gpu_moe import routing
from test_gpu_mxfp4 import DEV, packed

pytestmark = pytest.mark.gpu


def test_memory_freed_with_work_queued_is_not_written():
    """A tensor of the output's size is freed on the current stream while its last reader waits
    behind a few milliseconds of products; a call on another stream, not ordered after them, does
    not take its memory."""
    n = 4096
    xq, xs, _ = packed(n, 64, seed=1)
    wq, ws, _ = packed(n, 64, seed=2)
    want = b.mxfp4_gemm(xq, xs, wq, ws)
    big = torch.randn((4096, 4096), device=DEV)
    product = torch.empty_like(big)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    last = torch.full((n, n), 3.0, dtype=torch.bfloat16, device=DEV)
    for _ in range(8):
        torch.mm(big, big, out=product)
    copy = last.clone()
    address = last.data_ptr()
    del last
    out = b.mxfp4_gemm(xq, xs, wq, ws, stream=side)
    assert out.data_ptr() != address
    torch.cuda.synchronize()
    assert (copy == 3.0).all() and torch.equal(out, want)


def test_workspaces_and_dropped_outputs():
    """Chains on a side stream without buffers of the caller's, their intermediate results dropped as
    soon as the next call is queued, while the current stream allocates and writes tensors of the same sizes."""
    T, top, E, H, F = 300, 3, 6, 544, 288
    ids = torch.from_numpy(routing(T, top, E, seed=4, drop=0.05)).to(DEV)
    many = torch.from_numpy(routing(3000, top, E, seed=5, drop=0.05)).to(DEV)
    x = torch.randn((T, H), device=DEV).to(torch.bfloat16)
    weights = torch.rand((T, top), device=DEV)
    wq, ws, _ = packed(272, H, seed=1, lo=110, hi=124)
    w = []
    for n, k in ((2 * F, H), (H, F)):
        v = [packed(n, k, seed=20 + e, lo=116, hi=122) for e in range(E)]
        w += [torch.stack([t[0] for t in v]), torch.stack([t[1] for t in v])]

    def chain(stream):
        offsets, pos, token = b.moe_sort(ids, E, stream=stream)
        codes, scales = b.mxfp4_quantize_rows(x, stream=stream)
        hq, hs = b.mxfp4_expert_swiglu(codes, scales, offsets, w[0], w[1], row_token=token, stream=stream)
        rows = b.mxfp4_expert_gemm(hq, hs, offsets, w[2], w[3], stream=stream)
        return [b.moe_combine(rows, pos, weights, stream=stream), b.mxfp4_linear(x, wq, ws, stream=stream),
                b.mxfp4_moe(x, ids, weights, *w, stream=stream), *b.moe_sort(many, E, stream=stream)]

    want = chain(None)
    sizes = [b.mxfp4_linear_workspace(T, 272, H), b.moe_sort_workspace(9000, E), b.mxfp4_moe_workspace(T, top, E, H, F),
             *[t.numel() * t.element_size() for t in want]]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        got = chain(side)
        for size in sizes:
            torch.empty(size, dtype=torch.uint8, device=DEV).fill_(0xA5)
        torch.cuda.synchronize()
        assert all(torch.equal(g, v) for g, v in zip(got, want))
