"""The operators around a layer run together, as a model runs them: a feed-forward block between two norms, served in
16 bits, int8 and MXFP4 and trained in 16 bits; every step against its definition in 64 bits on the rows that the step
before wrote. The same run on a side stream, captured and replayed, and in the LDS-poisoned build, bit for bit."""
import os

import numpy as np
import pytest
import torch

import block_reference as ref
from gpu_layer import library
from quantized_gemm_quantize_amd import binding
from quantized_gemm_quantize_amd.build import POISON_LIB

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-5
H, F = 320, 608


def f64(t):
    return t.double().cpu().numpy()


def parameters(dtype, T, seed):
    rng = np.random.default_rng(seed)
    p = {}
    for name, shape, size in (("r", (T, H), 2.0), ("y", (T, H), 1.0), ("w1", (F, H), H ** -0.5), ("w2", (H, F), F ** -0.5),
                              ("d_out", (T, H), 1.0), ("d_new", (T, H), 1.0)):
        p[name] = ref.rounded(rng.standard_normal(shape) * size, dtype)[0].to(DEV)
    for name, n in (("weight", H), ("post", H), ("gate", H), ("weight2", H)):
        p[name] = torch.from_numpy(1 + 0.3 * rng.standard_normal(n)).float().to(DEV)
    for name, n in (("b1", F), ("b2", H)):
        p[name] = torch.from_numpy(rng.standard_normal(n)).float().to(DEV)
    p["q1"], p["s1"] = binding.w8a8_quantize_rows_f32(p["w1"].float())
    p["q2"], p["s2"] = binding.w8a8_quantize_rows_f32(p["w2"].float())
    p["c1"], p["e1"] = binding.mxfp4_quantize_rows(p["w1"])
    return p


def serve(p, b, stream=None):
    """16 bits, then int8, then the first step to MXFP4 rows."""
    k = dict(y=p["y"], post_weight=p["post"], gate=p["gate"], scale=0.5, eps=EPS, stream=stream)
    o = {}
    o["new"], o["n"] = b.block_norm(p["r"], p["weight"], **k)
    o["h"], o["pre"] = b.w16a16_linear(o["n"], p["w1"], bias=p["b1"], activation="gelu", pre=True, stream=stream)
    o["z"] = b.w16a16_linear(o["h"], p["w2"], bias=p["b2"], stream=stream)
    o["last"], o["out"] = b.block_norm(o["new"], p["weight2"], y=o["z"], eps=EPS, stream=stream)
    o["sum"] = b.w16a16_linear(o["h"], p["w2"], bias=p["b2"], residual=o["new"], stream=stream)
    if p["r"].dtype is torch.bfloat16:
        o["new8"], o["n8"], o["ns"] = b.block_norm_w8a8(p["r"], p["weight"], **k)
        o["h8"] = b.w8a8_gemm_act(o["n8"], o["ns"], p["q1"], p["s1"], bias=p["b1"], activation="gelu_tanh", stream=stream)
        o["hq"], o["hs"] = b.w8a8_quantize_rows(o["h8"], stream=stream)
        o["z8"] = b.w8a8_gemm_act(o["hq"], o["hs"], p["q2"], p["s2"], bias=p["b2"], residual=o["new8"], stream=stream)
        o["newx"], o["nx"], o["nxs"] = b.block_norm_mxfp4(p["r"], p["weight"], **k)
        o["hx"] = b.mxfp4_gemm(o["nx"], o["nxs"], p["c1"], p["e1"], stream=stream)
    return o


def train(p, o, b, stream=None):
    """The gradients of serve's 16-bit block: from out and last back to r, y and every parameter."""
    g = {}
    g["d_new2"], g["d_weight2"], g["d_z"], _, _ = b.block_norm_backward(p["d_out"], o["last"], p["weight2"], p["d_new"],
                                                                        y=o["z"], eps=EPS, stream=stream)
    g["d_h"], g["d_w2"], g["d_b2"], _ = b.w16a16_linear_backward(g["d_z"], o["h"], p["w2"], stream=stream)
    g["d_n"], g["d_w1"], g["d_b1"], g["d_pre"] = b.w16a16_linear_backward(g["d_h"], o["n"], p["w1"], pre=o["pre"],
                                                                          activation="gelu", stream=stream)
    g["d_r"], g["d_weight"], g["d_y"], g["d_post"], g["d_gate"] = b.block_norm_backward(
        g["d_n"], o["new"], p["weight"], g["d_new2"], y=p["y"], post_weight=p["post"], gate=p["gate"], scale=0.5, eps=EPS,
        stream=stream)
    return g


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T", [1, 37, 600])
def test_served(dtype, T):
    p = parameters(dtype, T, seed=T)
    o = serve(p, binding)
    v = {k: f64(t) for k, t in {**p, **o}.items()}
    new, e_new, n, e_n = ref.block_norm(v["r"], v["y"], True, v["post"], v["gate"], 0.5, v["weight"], EPS)
    ref.close(o["new"], new, e_new, dtype, "new")
    ref.close(o["n"], n, e_n, dtype, "n")
    pre, e_pre, h, e_h = ref.linear(v["n"], v["w1"], v["b1"], "gelu")
    ref.close(o["pre"], pre, e_pre, dtype, "pre")
    ref.close(o["h"], h, e_h, dtype, "h")
    _, _, z, e_z = ref.linear(v["h"], v["w2"], v["b2"])
    ref.close(o["z"], z, e_z, dtype, "z")
    last, e_last, out, e_out = ref.block_norm(v["new"], v["z"], weight=v["weight2"], eps=EPS)
    ref.close(o["last"], last, e_last, dtype, "last")
    ref.close(o["out"], out, e_out, dtype, "out")
    _, _, s, e_s = ref.linear(v["h"], v["w2"], v["b2"], residual=v["new"])
    ref.close(o["sum"], s, e_s, dtype, "sum")
    if dtype != "bf16":
        return
    assert torch.equal(o["new8"], o["new"]) and torch.equal(o["newx"], o["new"])
    # int8: exact integer products, the scales' two roundings, then the epilogue
    for x, s, w, sw, bias, a, res, got in (("n8", "ns", "q1", "s1", "b1", "gelu_tanh", None, "h8"),
                                           ("hq", "hs", "q2", "s2", "b2", "none", "new8", "z8")):
        acc = (v[x] @ v[w].T) * v[s][:, None] * v[sw][None, :]
        pre = acc + v[bias]
        e = 3 * ref.U * np.abs(acc) + ref.U * np.abs(pre)
        want = ref.act(pre, a)
        e = ref.STEEPEST * e + ref.ACT * np.abs(want) + ref.U * np.abs(pre) * (a != "none")
        if res:
            want = want + v[res]
            e = e + ref.U * np.abs(want)
        ref.close(o[got], want, e, dtype, got)
    x = f64(binding.mxfp4_dequantize_rows(o["nx"], o["nxs"], torch.float32))
    w = f64(binding.mxfp4_dequantize_rows(p["c1"], p["e1"], torch.float32))
    # each matrix instruction of 128 products rounds a sum, and the join of partial sums
    ref.close(o["hx"], x @ w.T, np.abs(x) @ np.abs(w).T * ((H / 64 + 8) * 2.0 ** -23), dtype, "hx")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T", [1, 37, 600])
def test_trained(dtype, T):
    p = parameters(dtype, T, seed=T + 1)
    o = serve(p, binding)
    g = train(p, o, binding)
    v = {k: f64(t) for k, t in {**p, **o, **g}.items()}
    want = ref.block_norm_backward(v["d_out"], v["d_new"], v["last"], v["z"], weight=v["weight2"], eps=EPS)
    for name, key, t in (("d_new2", "d_residual", dtype), ("d_weight2", "d_weight", "f32"), ("d_z", "d_y", dtype)):
        ref.close(g[name], *want[key], t, name)
    for d, x, w, d_x, d_w, d_b in (("d_z", "h", "w2", "d_h", "d_w2", "d_b2"), ("d_pre", "n", "w1", "d_n", "d_w1", None)):
        ref.close(g[d_x], *ref.product(v[d], np.ascontiguousarray(v[w].T)), dtype, d_x)
        ref.close(g[d_w], *ref.product(np.ascontiguousarray(v[d].T), np.ascontiguousarray(v[x].T)), dtype, d_w)
        if d_b:
            ref.close(g[d_b], v[d].sum(axis=0), ref.SUM * np.abs(v[d]).sum(axis=0), "f32", d_b)
    f = ref.slope(v["pre"], "gelu")
    d, e = v["d_h"] * f, np.abs(v["d_h"]) * (ref.SLOPE + ref.U * np.abs(f))
    ref.close(g["d_pre"], d, e, dtype, "d_pre")
    ref.close(g["d_b1"], d.sum(axis=0), (e + ref.SUM * np.abs(d)).sum(axis=0), "f32", "d_b1")
    want = ref.block_norm_backward(v["d_n"], v["d_new2"], v["new"], v["y"], True, v["post"], v["gate"], 0.5, v["weight"], EPS)
    for name, key, t in (("d_r", "d_residual", dtype), ("d_weight", "d_weight", "f32"), ("d_y", "d_y", dtype),
                         ("d_post", "d_post_weight", "f32"), ("d_gate", "d_gate", "f32")):
        ref.close(g[name], *want[key], t, name)


def everything(p, b, stream=None):
    o = serve(p, b, stream)
    return {**o, **train(p, o, b, stream)}


def same(got, want, what):
    for k in want:
        assert torch.equal(got[k].reshape(-1).view(torch.uint8), want[k].reshape(-1).view(torch.uint8)), f"{what}: {k}"


@pytest.mark.parametrize("T", [5, 600])
def test_side_stream(T):
    p = parameters("bf16", T, seed=3)
    want = everything(p, binding)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = everything(p, binding, stream=side)
    noise = [torch.full_like(t, 1) for t in want.values()]   # allocations of the same sizes meanwhile
    side.synchronize()
    same(got, want, "stream argument")
    with torch.cuda.stream(side):
        got = everything(p, binding)
    side.synchronize()
    same(got, want, "current stream")
    del noise


@pytest.mark.parametrize("T", [5, 600])
def test_captured(T):
    p = parameters("bf16", T, seed=4)
    want = everything(p, binding)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = everything(p, binding)
    for rep in range(4):
        for t in got.values():
            t.zero_()
        binding.block_norm(p["r"], p["weight2"])     # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        same(got, want, f"replay {rep}")


def test_two_graphs_share_a_workspace():
    """One workspace for two captured products with shared tiles and a norm's gradient: replayed in turn on one stream,
    each finds its own partial sums."""
    M, N, K = 72, 8, 4096
    sets = []
    work = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    need = [binding.w16a16_linear_workspace(M, N, K), binding.w16a16_linear_backward_workspace(600, N, K),
            binding.block_norm_backward_workspace(64, 320)]
    assert need[0] > 0 and max(need) <= work.numel()
    for seed in (1, 2):
        g = torch.Generator(device=DEV).manual_seed(seed)
        x, w = (torch.randn(s, generator=g, device=DEV).to(torch.bfloat16) for s in ((M, K), (N, K)))
        xs, d = (torch.randn(s, generator=g, device=DEV).to(torch.bfloat16) for s in ((600, K), (600, N)))
        r, o = (torch.randn((64, 320), generator=g, device=DEV) for _ in range(2))

        def run(x=x, w=w, xs=xs, d=d, r=r, o=o):
            return [binding.w16a16_linear(x, w, workspace=work), *binding.w16a16_linear_backward(d, xs, w, workspace=work)[:3],
                    *binding.block_norm_backward(o, r, workspace=work)[:2]]

        want = [t.clone() for t in run()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run()
        sets.append((graph, got, want, run))     # (run keeps the graph's inputs)
    for _ in range(3):
        for graph, *_ in sets:
            graph.replay()
        torch.cuda.synchronize()
        for _, got, want, _ in sets:
            assert all(torch.equal(a, c) for a, c in zip(got, want))
            for t in got:
                t.zero_()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T", [1, 20, 40, 64, 600, 2500])
def test_lds_poisoned(dtype, T):
    """No kernel reads what it has not written to LDS: a build that fills it first gives the same bits."""
    assert os.path.exists(POISON_LIB)
    p = parameters(dtype, T, seed=5)
    want = everything(p, binding)
    torch.cuda.synchronize()
    with library(POISON_LIB) as poisoned:
        got = everything(p, poisoned)
        torch.cuda.synchronize()
    same(got, want, "LDS-poisoned")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", [9, 65, 130, 517, 1031, 2056, 4099, 8200, 9001, 16384])
def test_lds_poisoned_norms(dtype, H):
    g = torch.Generator(device=DEV).manual_seed(H)
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    r, y, gate, d, n = (torch.randn((40, H), generator=g, device=DEV).to(t) for _ in range(5))

    def run(b):
        return [*b.block_norm(r, y=y, gate=gate, post_norm=True),
                *b.block_norm_backward(d, r, d_residual=n, y=y, gate=gate, post_norm=True),
                *(b.block_norm_w8a8(r) if H % 16 == 0 else ()), *(b.block_norm_mxfp4(r) if H % 32 == 0 else ())]

    want = run(binding)
    torch.cuda.synchronize()
    with library(POISON_LIB) as poisoned:
        got = run(poisoned)
        torch.cuda.synchronize()
    for a, c in zip(got, want):
        assert torch.equal(a.reshape(-1).view(torch.uint8), c.reshape(-1).view(torch.uint8))


@pytest.mark.parametrize("M,N,K", [(72, 8, 1024), (72, 8, 328), (200, 136, 3368), (768, 1408, 5080), (1608, 1944, 200), (1280, 720, 5640), (2192, 1352, 136), (3064, 2480, 1792),
                                   (2456, 3216, 344), (1504, 3536, 9544)])
def test_lds_poisoned_tiles(M, N, K):
    g = torch.Generator(device=DEV).manual_seed(K)
    x, w, d, w2 = (torch.randn(s, generator=g, device=DEV).to(torch.bfloat16) for s in ((M, K), (N, K), (M, K), (K, N)))
    dk, xk, wk = (torch.randn(s, generator=g, device=DEV).to(torch.bfloat16) for s in ((K, M), (K, N), (M, N)))
    x2 = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)

    def run(b):
        return [b.w16a16_linear(x, w, activation="silu"), b.w16a16_linear_backward(d, x2, w2, d_w=False, d_bias=False)[0],
                b.w16a16_linear_backward(dk, xk, wk, d_x=False, d_bias=False)[1]]

    want = run(binding)
    torch.cuda.synchronize()
    with library(POISON_LIB) as poisoned:
        got = run(poisoned)
        torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))


@pytest.mark.parametrize("M,N,K", [(2, 992, 8), (331, 2224, 8), (333, 8, 8), (3547, 4744, 72), (982, 8, 8), (8, 8, 8), (128, 2328, 1000), (1964, 72, 1240), (2008, 1816, 2144),
                                   (1343, 7600, 656), (934, 776, 4808), (3855, 1000, 2272)])
def test_lds_poisoned_gradients(M, N, K):
    """Both in one launch."""
    g = torch.Generator(device=DEV).manual_seed(K)
    d, x, w = (torch.randn(s, generator=g, device=DEV).to(torch.bfloat16) for s in ((M, N), (M, K), (N, K)))
    want = binding.w16a16_linear_backward(d, x, w)
    torch.cuda.synchronize()
    with library(POISON_LIB) as poisoned:
        got = poisoned.w16a16_linear_backward(d, x, w)
        torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", [520, 1031, 5000, 9000, 9001, 16384])
def test_gradients_in_place(dtype, H):
    """d_residual over d_new or d_out, d_y over y, d_gate over the gate's rows: what the header allows, through the
    library, with rows held in registers and rows read again."""
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    code = binding.MXFP4_F32 if dtype == "f32" else binding.MXFP4_BF16
    g = torch.Generator(device=DEV).manual_seed(H)
    T = 300
    d, n, r, y, gate = (torch.randn((T, H), generator=g, device=DEV).to(t) for _ in range(5))
    want = binding.block_norm_backward(d, r, d_residual=n, y=y, gate=gate, post_norm=True, eps=EPS)
    lib = binding.load()
    need = binding.block_norm_backward_workspace(T, H)
    for over in ("d", "n"):
        c = {k: v.clone() for k, v in dict(d=d, n=n, y=y, gate=gate).items()}
        vectors = torch.empty((2, -(-H // 4) * 4), device=DEV)
        work = torch.empty(need, dtype=torch.uint8, device=DEV)
        status = lib.block_norm_backward(c["d"].data_ptr(), H, c["n"].data_ptr(), H, r.data_ptr(), H, c["y"].data_ptr(), H, 1, None,
                                         c["gate"].data_ptr(), H, 1.0, None, EPS, T, H, code, c[over].data_ptr(), c["y"].data_ptr(),
                                         c["gate"].data_ptr(), vectors[0].data_ptr(), vectors[1].data_ptr(), work.data_ptr(), need,
                                         torch.cuda.current_stream().cuda_stream)
        assert status == binding.W8A8_OK
        torch.cuda.synchronize()
        got = (c[over], vectors[0, :H], c["y"], vectors[1, :H], c["gate"])
        for i, (a, e) in enumerate(zip(got, want)):
            assert torch.equal(a, e), (over, i)
