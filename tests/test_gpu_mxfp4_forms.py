"""MXFP4 products through every compiled variant of their kernels, ragged groups, empty experts and
dropped slots among them, against 64 bits."""
import os

import numpy as np
import pytest
import torch

import mx_reference as ref
from gpu_layer import library
from mxfp4_sizes import DENSE, DEPTHS, GROUPED
from quantized_gemm_quantize_amd import binding as b
from quantized_gemm_quantize_amd import build
from test_gpu_moe import check_hidden, routing
from test_gpu_mxfp4 import DEV, HALF_ULP, TINY, TYPES, packed, rows

pytestmark = pytest.mark.gpu


def storage(lead, n, k, lo, hi, seed):
    """Random MXFP4 storage [*lead, n, k] on the GPU, padded scales 0."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    codes = torch.randint(0, 256, (*lead, n, k // 2), generator=g, device=DEV).to(torch.uint8)
    scales = torch.randint(lo, hi, (*lead, -(-k // 256), n, 8), generator=g, device=DEV).to(torch.uint8)
    if k % 256:
        scales[..., -1, :, k % 256 // 32:] = 0
    return codes, scales


def values(codes, scales):
    """In float64 (the dequantization is exact)."""
    return b.mxfp4_dequantize_rows(codes, scales, torch.float32).double()


def plan(T, top, E, seed):
    """Ragged groups: every third expert has no slot, some slots no expert."""
    rng = np.random.default_rng(seed)
    ids = rng.permuted(np.tile(np.arange(E), (T, 1)), axis=1)[:, :top]
    ids = np.where((ids % 3 == 2) & (E > 4), np.where(rng.random((T, top)) < 0.8, ids - 1, ids - 2), ids)
    ids[rng.random((T, top)) < 0.03] = -1
    offsets, _, token = ref.sort(ids, E)
    return offsets, token, torch.from_numpy(offsets).to(DEV), torch.from_numpy(token).to(DEV)


def product(x, w):
    """(x w^T, the bound of an fp32 product's error): exact products, K / 64 + 8 roundings of a
    partial sum."""
    want, mag = x @ w.t().contiguous(), x.abs() @ w.abs().t().contiguous()
    return want, mag * ((x.shape[1] / 64 + 8) * 2.0 ** -23)


@pytest.mark.parametrize("K", DEPTHS)
@pytest.mark.parametrize("T,top,E,N", GROUPED)
def test_grouped(T, top, E, N, K):
    offsets, token, offsets_t, token_t = plan(T, top, E, seed=T + K)
    S = T * top
    xq, xs = storage((), T, K, 122, 126, seed=1)
    wq, ws = storage((E,), N, K, 120, 124, seed=2)
    outs = {d: b.mxfp4_expert_gemm(xq, xs, offsets_t, wq, ws, row_token=token_t, out_dtype=t,
                                   out=torch.full((S, N), 7.0, dtype=t, device=DEV)) for d, t in TYPES.items()}
    hq = torch.full((S, N // 4), 0x77, dtype=torch.uint8, device=DEV)
    hs = torch.full((-(-N // 512), S, 8), 0x77, dtype=torch.uint8, device=DEV)
    b.mxfp4_expert_swiglu(xq, xs, offsets_t, wq, ws, row_token=token_t, hq=hq, hs=hs)
    xv = values(xq, xs)
    h, slack = np.zeros((S, N // 2)), np.zeros((S, N // 2))
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        if lo == hi:
            continue
        gu, err = product(xv[torch.from_numpy(token[lo:hi]).to(DEV).long()], values(wq[e], ws[e]))
        for d, out in outs.items():
            bound = err + gu.abs() * (HALF_ULP[d] * 1.001) + TINY[d]
            assert ((out[lo:hi].double() - gu).abs() <= bound).all(), (d, e)
        gu, err = gu.cpu().numpy(), err.cpu().numpy()
        h[lo:hi] = ref.swiglu(gu)
        # |d silu| <= 1.1, |silu(g)| <= |g|; the activation's own roundings are below 2^-20 together
        slack[lo:hi] = (1.1 * err[:, 0::2] * np.abs(gu[:, 1::2]) + err[:, 1::2] * np.abs(gu[:, 0::2])
                        + np.abs(h[lo:hi]) * 2.0 ** -20)
    for out in outs.values():
        assert (out[offsets[E]:] == 0).all()
    check_hidden(hq, hs, h, slack)
    assert (hq[offsets[E]:] == 0).all() and (hs[:, offsets[E]:] == 0).all()


@pytest.mark.parametrize("K", DEPTHS)
@pytest.mark.parametrize("M,N", DENSE)
def test_dense(M, N, K):
    xq, xs = storage((), M, K, 118, 126, seed=1)
    wq, ws = storage((), N, K, 118, 126, seed=2)
    want, err = product(values(xq, xs), values(wq, ws))
    for d, t in TYPES.items():
        bound = err + want.abs() * (HALF_ULP[d] * 1.001) + TINY[d]
        assert ((b.mxfp4_gemm(xq, xs, wq, ws, out_dtype=t).double() - want).abs() <= bound).all(), d


def test_all_rows_on_one_expert():
    """The kernel is chosen from the average; with every slot on one of many experts, its rows run through
    the same workgroups one after another."""
    for T, E, N, K in ((600, 64, 768, 544), (1200, 64, 768, 544), (2000, 8, 704, 1312)):
        xq, xs = storage((), T, K, 122, 126, seed=1)
        wq, ws = storage((E,), N, K, 120, 124, seed=2)
        offsets, _, token = b.moe_sort(torch.full((T, 1), E - 2, dtype=torch.int64, device=DEV), E)
        out = b.mxfp4_expert_gemm(xq, xs, offsets, wq, ws, row_token=token, out_dtype=torch.float32)
        want, err = product(values(xq, xs), values(wq[E - 2], ws[E - 2]))
        assert ((out.double() - want).abs() <= err + want.abs() * (HALF_ULP["f32"] * 1.001) + TINY["f32"]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,top,E,H,F", [(1, 4, 8, 2080, 288), (2, 4, 8, 2080, 288), (1, 4, 8, 1056, 288), (1, 8, 8, 2080, 2080)])
def test_few_slots_of_wide_tokens(T, top, E, H, F, dtype):
    """The gate and up products of a few slots by 8 wavefronts (H from 1793 on, as many workgroups as
    compute units at most) and by 4: each slot's own experts, in 64 bits. Hidden elements within the fp32 error
    of a rounding boundary may land on its other side (2^-9.5 of the norm)."""
    ids = torch.from_numpy(routing(T, top, E, seed=T)).to(DEV)
    weights = torch.rand((T, top), generator=torch.Generator().manual_seed(1)).to(DEV)
    x, x64 = rows(T, H, dtype, seed=2, spread=0.5)
    w13q, w13s = storage((E,), 2 * F, H, 119, 123, seed=3)
    w2q, w2s = storage((E,), H, F, 119, 123, seed=4)
    out = b.mxfp4_moe(x, ids, weights, w13q, w13s, w2q, w2s)
    xv = ref.values(*ref.quantize(x64))
    want = np.zeros((T, H))
    for t, slots in enumerate(ids.tolist()):
        for j, e in enumerate(slots):
            h = ref.values(*ref.quantize(ref.swiglu(xv[t:t + 1] @ values(w13q[e], w13s[e]).cpu().numpy().T)))
            want[t] += weights[t, j].item() * (h @ values(w2q[e], w2s[e]).cpu().numpy().T)[0]
    err = np.linalg.norm(out.double().cpu().numpy() - want)
    assert err <= (2.0 ** -8 + 2 * HALF_ULP[dtype]) * np.linalg.norm(want)


def test_lds_poisoned_build_gives_the_same():
    """Every variant again in the build whose kernels fill their LDS with a pattern first: a read of LDS
    that the launch has not written would change the bits."""
    if not os.path.exists(build.POISON_LIB):
        pytest.skip("the LDS-poisoned build is missing")
    ks = (64, 288, 512, 768, 1312)
    cases = []
    for T, top, E, N in GROUPED:
        _, _, offsets, token = plan(T, top, E, seed=T)
        for K in ks:
            cases.append((storage((), T, K, 122, 126, seed=1), offsets, storage((E,), N, K, 120, 124, seed=2), token))
    dense = [(storage((), M, K, 118, 126, seed=1), storage((), N, K, 118, 126, seed=2)) for M, N in DENSE for K in ks]

    def run():
        out = []
        for x, offsets, w, token in cases:
            out.append(b.mxfp4_expert_gemm(*x, offsets, *w, row_token=token))
            out += b.mxfp4_expert_swiglu(*x, offsets, *w, row_token=token)
        return out + [b.mxfp4_gemm(*x, *w) for x, w in dense]

    want = run()
    torch.cuda.synchronize()
    with library(build.POISON_LIB):
        got = run()
        torch.cuda.synchronize()
    for g, v in zip(got, want):
        assert torch.equal(g.view(torch.uint8), v.view(torch.uint8))
