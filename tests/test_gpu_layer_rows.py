"""The expert layer's rows between its products and its weighted sum: what their type costs."""
import pytest
import torch

from quantized_gemm_quantize_amd import binding as b
from test_gpu_moe import routing
from test_gpu_mxfp4 import DEV, HALF_ULP, TINY, TYPES, packed, rows

pytestmark = pytest.mark.gpu


def stacks(E, H, F, lo=119, hi=123):
    out = []
    for n, k, seed in ((2 * F, H, 10), (H, F, 50)):
        w = [packed(n, k, seed=seed + e, lo=lo, hi=hi) for e in range(E)]
        out += [torch.stack([v[0] for v in w]), torch.stack([v[1] for v in w])]
    return out


def parts(x, ids, weights, w13q, w13s, w2q, w2s):
    """(the experts' rows in fp32, their positions) of the layer's own operators."""
    offsets, slot_pos, row_token = b.moe_sort(ids, w13q.shape[0])
    xq, xs = b.mxfp4_quantize_rows(x)
    hq, hs = b.mxfp4_expert_swiglu(xq, xs, offsets, w13q, w13s, row_token=row_token)
    return b.mxfp4_expert_gemm(hq, hs, offsets, w2q, w2s, out_dtype=torch.float32), slot_pos


@pytest.mark.parametrize("T,top,E,H,F,drop", [(64, 4, 32, 256, 96, 0.0), (20, 5, 8, 288, 160, 0.1), (257, 2, 5, 1312, 736, 0.05),
                                              (1100, 3, 4, 544, 288, 0.0)])
def test_bf16_layer_rounds_once(T, top, E, H, F, drop):
    """A bfloat16 layer is the fp32 weighted sum of its experts' fp32 rows, rounded once: at most
    half a unit in the last place from the sum in 64 bits of those rows, beside the sum's own roundings (2 top
    of 2^-24 of the magnitudes)."""
    ids = torch.from_numpy(routing(T, top, E, seed=T, drop=drop)).to(DEV)
    weights = torch.rand((T, top), generator=torch.Generator().manual_seed(1)).to(DEV)
    x, _ = rows(T, H, "bf16", seed=2, spread=0.5)
    w = stacks(E, H, F)
    out = b.mxfp4_moe(x, ids, weights, *w).double()
    y, pos = parts(x, ids, weights, *w)
    assert torch.equal(out, b.moe_combine(y, pos, weights).to(torch.bfloat16).double())
    kept = (pos >= 0).unsqueeze(2)
    terms = torch.where(kept, y.double()[pos.clamp_min(0).long()] * weights.double().unsqueeze(2), 0.0)
    want, mag = terms.sum(dim=1), terms.abs().sum(dim=1)
    bound = want.abs() * (HALF_ULP["bf16"] * 1.001) + mag * ((2 * top + 1) * 2.0 ** -24) + TINY["bf16"]
    assert ((out - want).abs() <= bound).all()


@pytest.mark.parametrize("T,top", [(2, 2), (60, 2)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_sums_within_the_type_are_finite(T, top, dtype):
    """Experts' outputs beyond binary16's largest value whose weighted sum lies within it: the same
    in the form for a few slots and the sorted one (H * F is too large for few slots at T = 60)."""
    E, H, F = 3, 2048, 256
    x = torch.ones((T, H), dtype=TYPES[dtype], device=DEV)
    # gates and ups: 2048 products of 1 and 2^-11, i.e. 1; down: 256 units of silu(1) * 1, times 2^9
    q = lambda *shape: torch.full(shape, 0x22, dtype=torch.uint8, device=DEV)
    scales = lambda value, *shape: torch.full(shape, value, dtype=torch.uint8, device=DEV)
    w13 = q(E, 2 * F, H // 2), scales(127 - 11, E, H // 256, 2 * F, 8)
    w2 = q(E, H, F // 2), scales(127 + 9, E, F // 256, H, 8)
    ids = torch.arange(T * top, device=DEV).reshape(T, top) % E
    weights = torch.full((T, top), 0.125, device=DEV)
    out = b.mxfp4_moe(x, ids, weights, *w13, *w2)
    want = top * 0.125 * 256 * 512 * 0.75
    assert 256 * 512 * 0.75 > 65504 > want        # silu(1) = 0.731 has the 4-bit value 0.75
    assert (out.double() == want).all()
