"""MXFP4 products at sizes that reach every kernel, with every count of K stages, offsets past 32
bits, other streams, captured graphs, repeated runs and the LDS-poisoned build."""
import os

import numpy as np
import pytest
import torch

import mx_reference as ref
from gpu_layer import library
from quantized_gemm_quantize_amd import binding as b
from quantized_gemm_quantize_amd import build
from test_gpu_moe import check_hidden, routing
from test_gpu_mxfp4 import DEV, HALF_ULP, packed

pytestmark = pytest.mark.gpu


def gpu_values(codes, scales):
    """The values of MXFP4 storage in float64 on the GPU (the dequantization is exact)."""
    return b.mxfp4_dequantize_rows(codes, scales, torch.float32).double()


def check_on_gpu(got, x, w, dtype="f32"):
    """As check_product: exact products, K / 64 + 8 roundings of a partial sum, one of the result."""
    want, mag = x @ w.t().contiguous(), x.abs() @ w.abs().t().contiguous()
    bound = mag * ((x.shape[1] / 64 + 8) * 2.0 ** -23) + want.abs() * (HALF_ULP[dtype] * 1.001) + 1e-37
    assert ((got.double() - want).abs() <= bound).all()


# rows and channels whose 64x64, 64x128, 128x128 and 256x128 tiles are the first that run at once on
# 256 CUs, more than that with short and with long K, and the weight-streaming ones (16, 32, 64 rows)
TILES = [(7, 144), (31, 272), (50, 1040), (200, 4112), (390, 4112), (700, 4112), (1500, 4112), (4100, 4112)]


@pytest.mark.parametrize("m,n", TILES)
@pytest.mark.parametrize("k", [32, 128, 256, 288, 544, 800, 1024, 1056, 1312, 1568, 2080])
def test_every_tile_and_stage_count(m, n, k):
    xq, xs, _ = packed(m, k, seed=m)
    wq, ws, _ = packed(n, k, seed=k, lo=110, hi=130)
    check_on_gpu(b.mxfp4_gemm(xq, xs, wq, ws, out_dtype=torch.float32), gpu_values(xq, xs), gpu_values(wq, ws))


@pytest.mark.parametrize("T,top,E,F,K", [(3000, 2, 4, 1088, 288), (3000, 2, 4, 1088, 544), (2100, 3, 6, 544, 1312),
                                         (1100, 2, 2, 288, 800), (400, 2, 3, 288, 544), (2500, 8, 100, 64, 96),
                                         (16000, 1, 500, 32, 64)])
def test_swiglu_tiles(T, top, E, F, K):
    """Groups of many rows (the tiled kernel takes several tiles per workgroup), ragged, some empty."""
    ids = routing(T, top, E, seed=T, drop=0.03)
    offsets, _, row_token = ref.sort(ids, E)
    xq, xs, _ = packed(T, K, seed=K, lo=122, hi=128)
    w = [packed(2 * F, K, seed=100 + e, lo=118, hi=124) for e in range(E)]
    hq, hs = b.mxfp4_expert_swiglu(xq, xs, torch.from_numpy(offsets).to(DEV), torch.stack([v[0] for v in w]),
                                   torch.stack([v[1] for v in w]), row_token=torch.from_numpy(row_token).to(DEV))
    h, slack = np.zeros((T * top, F)), np.zeros((T * top, F))
    xv = gpu_values(xq, xs)
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        if lo == hi:
            continue
        xe, we = xv[torch.from_numpy(row_token[lo:hi]).to(DEV).long()], gpu_values(w[e][0], w[e][1])
        gu = (xe @ we.t().contiguous()).cpu().numpy()
        err = (xe.abs() @ we.abs().t().contiguous()).cpu().numpy() * (K / 64 + 8) * 2.0 ** -23
        h[lo:hi] = ref.swiglu(gu)
        slack[lo:hi] = (1.1 * err[:, 0::2] * np.abs(gu[:, 1::2]) + err[:, 1::2] * np.abs(gu[:, 0::2])
                        + np.abs(h[lo:hi]) * 2.0 ** -20)
    check_hidden(hq, hs, h, slack)


@pytest.mark.parametrize("T,top,E,N,K", [(4000, 2, 3, 2064, 800), (4000, 2, 3, 2064, 1312), (500, 2, 40, 272, 1056)])
def test_expert_gemm_tiles(T, top, E, N, K):
    ids = routing(T, top, E, seed=T, drop=0.03)
    offsets, _, _ = ref.sort(ids, E)
    xq, xs, _ = packed(T * top, K, seed=K)
    w = [packed(N, K, seed=100 + e, lo=110, hi=130) for e in range(E)]
    out = b.mxfp4_expert_gemm(xq, xs, torch.from_numpy(offsets).to(DEV), torch.stack([v[0] for v in w]),
                              torch.stack([v[1] for v in w]), out_dtype=torch.float32)
    xv = gpu_values(xq, xs)
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        if lo < hi:
            check_on_gpu(out[lo:hi], xv[lo:hi], gpu_values(w[e][0], w[e][1]))
    assert (out[offsets[E]:] == 0).all()


def test_outputs_past_32_bits():
    """More than 2^31 outputs, and codes past 2^32 bytes of values: rows at both ends are right."""
    m, n, k = 525000, 4112, 64
    xq, xs, _ = packed(m, k, seed=1)
    wq, ws, _ = packed(n, k, seed=2)
    out = b.mxfp4_gemm(xq, xs, wq, ws)
    for lo in (0, 262143, m - 100):
        x = gpu_values(xq[lo:lo + 100], xs[:, lo:lo + 100].clone())
        check_on_gpu(out[lo:lo + 100], x, gpu_values(wq, ws), "bf16")
    del out
    values = b.mxfp4_dequantize_rows(torch.full((140000, 8192), 0x21, dtype=torch.uint8, device=DEV),
                                     torch.full((64, 140000, 8), 127, dtype=torch.uint8, device=DEV), torch.bfloat16)
    assert values.numel() > 2 ** 31
    assert (values[-3:, 0::2] == 0.5).all() and (values[-3:, 1::2] == 1.0).all()
    codes, scales = b.mxfp4_quantize_rows(values)
    assert (codes[-3:] == 0x64).all() and (scales[:, -3:] == 125).all()


def test_rows_past_32_bits():
    T, top, H = 140000, 4, 4104
    ids = (torch.arange(T * top, device=DEV) * 7919 % 8).reshape(T, top)
    offsets, slot_pos, _ = b.moe_sort(ids, 8)
    x = torch.randn((T, 8), device=DEV).repeat(1, H // 8).to(torch.bfloat16)
    rows = b.moe_gather(x, slot_pos)
    assert rows.numel() > 2 ** 31
    at = torch.tensor([0, T // 2, T - 1], device=DEV)
    for j in range(top):
        assert torch.equal(rows[slot_pos[at, j].long()], x[at])
    w = torch.full((T, top), 0.25, device=DEV)
    assert torch.equal(b.moe_combine(rows, slot_pos, w), x)
    d_rows, d_w = b.moe_combine_backward(x, rows, slot_pos, w)
    assert torch.equal(d_rows[slot_pos[at, 1].long()], (x[at].float() * 0.25).to(torch.bfloat16))


# ------------------------------------------------------------------ whole runs

def make_set():
    g = torch.Generator(device=DEV).manual_seed(3)
    t = {"x": torch.randn((300, 544), generator=g, device=DEV).to(torch.bfloat16),
         "weights": torch.rand((300, 3), generator=g, device=DEV),
         "ids": torch.from_numpy(routing(300, 3, 6, seed=4, drop=0.05)).to(DEV)}
    t["wq"], t["ws"], _ = packed(272, 544, seed=1, lo=110, hi=124)
    for name, n, k in (("w13", 2 * 288, 544), ("w2", 544, 288)):
        w = [packed(n, k, seed=20 + e, lo=116, hi=122) for e in range(6)]
        t[name + "q"], t[name + "s"] = torch.stack([v[0] for v in w]), torch.stack([v[1] for v in w])
    t["y"] = torch.randn((900, 544), generator=g, device=DEV).to(torch.bfloat16)
    t["many"] = torch.from_numpy(routing(3000, 3, 6, seed=5, drop=0.05)).to(DEV)
    t["work"] = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    return t


def run_set(t, stream=None):
    """Every entry point once."""
    o = {}
    o["codes"], o["scales"] = b.mxfp4_quantize_rows(t["x"], stream=stream)
    o["values"] = b.mxfp4_dequantize_rows(o["codes"], o["scales"], stream=stream)
    o["gemm"] = b.mxfp4_gemm(o["codes"], o["scales"], t["wq"], t["ws"], stream=stream)
    for m in (1, 4, 20, 50, 300):
        o["linear%d" % m] = b.mxfp4_linear(t["x"][:m], t["wq"], t["ws"], workspace=t["work"], stream=stream)
    o["offsets"], o["pos"], o["token"] = b.moe_sort(t["ids"], 6, stream=stream)
    o["o2"], o["p2"], o["t2"] = b.moe_sort(t["many"], 6, workspace=t["work"], stream=stream)
    o["rows"] = b.moe_gather(t["x"], o["pos"], stream=stream)
    o["comb"] = b.moe_combine(t["y"], o["pos"], t["weights"], stream=stream)
    o["d_rows"], o["d_w"] = b.moe_combine_backward(t["x"], t["y"], o["pos"], t["weights"], stream=stream)
    o["d_x"] = b.moe_gather_backward(t["y"], o["pos"], stream=stream)
    o["hq"], o["hs"] = b.mxfp4_expert_swiglu(o["codes"], o["scales"], o["offsets"], t["w13q"], t["w13s"],
                                             row_token=o["token"], stream=stream)
    o["down"] = b.mxfp4_expert_gemm(o["hq"], o["hs"], o["offsets"], t["w2q"], t["w2s"], stream=stream)
    for m in (1, 2, 16, 300):
        o["moe%d" % m] = b.mxfp4_moe(t["x"][:m], t["ids"][:m].contiguous(), t["weights"][:m].contiguous(),
                                     t["w13q"], t["w13s"], t["w2q"], t["w2s"], workspace=t["work"], stream=stream)
    return o


def same(a, c):
    return all(torch.equal(a[k].view(torch.uint8), c[k].view(torch.uint8)) for k in a)


def test_runs_repeat_bit_for_bit():
    t = make_set()
    first = run_set(t)
    for _ in range(9):
        assert same(run_set(t), first)


def test_other_stream():
    t = make_set()
    want = run_set(t)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run_set(t, stream=s)
    s.synchronize()
    assert same(got, want)
    with torch.cuda.stream(s):
        inside = run_set(t)
    s.synchronize()
    assert same(inside, want)


def test_graph_replays():
    t = make_set()
    want = run_set(t)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run_set(t)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = run_set(t)
    for i in range(5):
        for v in got.values():
            v.view(torch.uint8).fill_(0xA5)
        run_set(t)                                           # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want), i


def test_lds_poisoned_build_gives_the_same():
    if not os.path.exists(build.POISON_LIB):
        pytest.skip("the LDS-poisoned build is missing")
    t = make_set()
    big = [packed(4100, 544, seed=1), packed(4112, 544, seed=2), packed(1500, 1312, seed=3), packed(4112, 1312, seed=4)]

    def products():
        return {"short": b.mxfp4_gemm(*big[0][:2], *big[1][:2]), "mid": b.mxfp4_gemm(*big[2][:2], *big[3][:2]),
                "long": b.mxfp4_gemm(*big[3][:2], *big[3][:2])}

    want, want_big = run_set(t), products()
    torch.cuda.synchronize()
    for _ in range(2):
        with library(build.POISON_LIB):
            got, got_big = run_set(t), products()
            torch.cuda.synchronize()
        assert same(got, want) and same(got_big, want_big)
        assert same(run_set(t), want)


def test_a_plan_of_any_numbers_stays_in_bounds():
    """Offsets and positions that no sort made: unspecified values, but nothing outside the outputs
    is written (guard rows around them keep their pattern)."""
    g = torch.Generator(device=DEV).manual_seed(9)
    T, top, E, H = 40, 3, 5, 288
    x = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
    y = torch.randn((T * top, H), generator=g, device=DEV).to(torch.bfloat16)
    wq, ws, _ = packed(64, H, seed=1)
    xq, xs = b.mxfp4_quantize_rows(x)
    weights = torch.rand((T, top), generator=g, device=DEV)

    def guarded(rows, width, dtype):
        full = torch.full((rows + 32, width), 7, dtype=dtype, device=DEV)
        return full, full[16:16 + rows]

    for _ in range(4):
        pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (T, top), generator=g, device=DEV).to(torch.int32)
        pos[::3] = torch.randint(-200, 200, pos[::3].shape, generator=g, device=DEV).to(torch.int32)
        offsets = torch.randint(-300, 300, (E + 1,), generator=g, device=DEV).to(torch.int32)
        token = torch.randint(-2 ** 31, 2 ** 31 - 1, (T * top,), generator=g, device=DEV).to(torch.int32)
        outs = [guarded(T * top, H, torch.bfloat16), guarded(T, H, torch.bfloat16), guarded(T * top, H, torch.bfloat16),
                guarded(T * top, 64, torch.float32)]
        b.moe_gather(x, pos, out=outs[0][1])
        b.moe_combine(y, pos, weights, out=outs[1][1])
        b.moe_combine_backward(x, y, pos, weights, d_rows=outs[2][1])
        b.mxfp4_expert_gemm(xq, xs, offsets, wq.expand(E, 64, H // 2).contiguous(),
                            ws.expand(E, 2, 64, 8).contiguous(), row_token=token, out=outs[3][1],
                            out_dtype=torch.float32)
        torch.cuda.synchronize()
        for full, _ in outs:
            assert (full[:16] == 7).all() and (full[-16:] == 7).all()
