"""Mixture-of-experts routing and the experts' MXFP4 products against their definitions in 64 bits."""
import numpy as np
import pytest
import torch

import mx_reference as ref
from quantized_gemm_quantize_amd import binding as b
from test_gpu_mxfp4 import DEV, HALF_ULP, TINY, TYPES, check_product, packed, rows

pytestmark = pytest.mark.gpu


def routing(T, top, E, seed, drop=0.0, skew=False):
    """Distinct experts per token (uniform, or nearly all tokens on few experts), dropped slots."""
    rng = np.random.default_rng(seed)
    logits = rng.standard_normal((T, E)) + (4.0 * (np.arange(E) < top) if skew else 0.0)
    ids = np.argsort(-logits, axis=1)[:, :top]
    ids[rng.random((T, top)) < drop] = -1
    return ids


PLANS = [(1, 1, 1, 0.0), (1, 4, 32, 0.0), (3, 2, 8, 0.5), (64, 4, 32, 0.0), (129, 2, 8, 0.1),
         (700, 6, 17, 0.05), (1025, 4, 512, 0.0), (2049, 2, 64, 0.3), (5000, 8, 130, 0.02)]


@pytest.mark.parametrize("T,top,E,drop", PLANS)
@pytest.mark.parametrize("wide", [False, True])
def test_sort(T, top, E, drop, wide):
    ids = routing(T, top, E, seed=T, drop=drop)
    t = torch.from_numpy(ids).to(torch.int64 if wide else torch.int32).to(DEV)
    offsets, slot_pos, row_token = b.moe_sort(t, E)
    want = ref.sort(ids, E)
    assert np.array_equal(offsets.cpu().numpy(), want[0])
    assert np.array_equal(slot_pos.cpu().numpy(), want[1])
    assert np.array_equal(row_token.cpu().numpy(), want[2])


@pytest.mark.parametrize("T,top,E", [(30000, 8, 512), (12300, 4, 511), (50000, 8, 130), (1100000, 4, 100), (70000, 8, 3)])
def test_sort_many_slots(T, top, E):
    """Slots of many workgroups, whose counts each sums or a scan does (one and two passes of it)."""
    ids = np.random.default_rng(E).integers(-1, E + 1, (T, top))
    ids[T // 3:T // 2] = E - 1  # workgroups with a single expert
    got = b.moe_sort(torch.from_numpy(ids).to(DEV), E)
    for g, w in zip(got, ref.sort(ids, E)):
        assert np.array_equal(g.cpu().numpy(), w)


def test_sort_ids_outside_the_experts():
    """Any id outside [0, E) is a dropped slot, 64-bit ones that wrap in 32 bits too."""
    ids = np.array([[0, 7, 8], [-1, 2 ** 32 + 3, -2 ** 63], [3, 2 ** 31, 3], [2 ** 63 - 1, 1, 0]])
    got = b.moe_sort(torch.from_numpy(ids).to(DEV), 8)
    for g, w in zip(got, ref.sort(ids, 8)):
        assert np.array_equal(g.cpu().numpy(), w)


def test_sort_edges():
    """No token; all slots on one expert; none kept."""
    none = torch.empty((0, 2), dtype=torch.int32, device=DEV)
    assert b.moe_sort(none, 5)[0].tolist() == [0] * 6
    for value in (4, 9):
        ids = np.full((3000, 3), value)
        got = b.moe_sort(torch.from_numpy(ids).to(DEV), 5)
        for g, w in zip(got, ref.sort(ids, 5)):
            assert np.array_equal(g.cpu().numpy(), w)


ROWS = [(1, 1, 1, 1, 0.0), (1, 4, 8, 4096, 0.0), (9, 2, 4, 33, 0.3), (17, 3, 5, 8, 0.2),
        (64, 8, 64, 1031, 0.1), (130, 2, 8, 2056, 0.0), (33, 11, 16, 264, 0.4)]


def close(got, want, mag, terms, dtype):
    """Each of `terms` products and sums rounds to 2^-24 of the magnitudes at worst; then one
    rounding to the type."""
    bound = (terms + 1) * 2.0 ** -24 * mag + np.abs(want) * HALF_ULP[dtype] * 1.001 + TINY[dtype]
    assert (np.abs(got.double().cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,top,E,H,drop", ROWS)
def test_rows_and_back(T, top, E, H, drop, dtype):
    rng = np.random.default_rng(T * H)
    _, pos, _ = ref.sort(routing(T, top, E, seed=H, drop=drop), E)
    pos_t = torch.from_numpy(pos).to(DEV)

    def tensor(*shape):
        t = torch.from_numpy(rng.standard_normal(shape)).to(TYPES[dtype])
        return t.to(DEV), t.double().numpy()

    x, x64 = tensor(T, H)
    got = b.moe_gather(x, pos_t)
    assert np.array_equal(got.double().cpu().numpy(), ref.gather(x64, pos))
    y, y64 = tensor(T * top, H)
    w = rng.random((T, top)).astype(np.float32)
    w_t = torch.from_numpy(w).to(DEV)
    want, mag = ref.combine(y64, pos, w.astype(np.float64))
    close(b.moe_combine(y, pos_t, w_t), want, mag, 2 * top, dtype)
    want, mag = ref.combine(y64, pos)
    close(b.moe_gather_backward(y, pos_t), want, mag, top, dtype)
    d, d64 = tensor(T, H)
    d_rows, d_w = b.moe_combine_backward(d, y, pos_t, w_t)
    want_r, want_w, mag_w = ref.combine_backward(d64, y64, pos, w.astype(np.float64))
    close(d_rows, want_r, np.abs(want_r), 1, dtype)
    # a sum over H in a tree: at most H / 256 + 16 roundings in a row, each product one more
    bound = (H / 256 + 18) * 2.0 ** -24 * mag_w + 1e-40
    assert (np.abs(d_w.double().cpu().numpy() - want_w) <= bound).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dropped_slots_take_nothing(dtype):
    """Infinities and NaN in the rows and weights of dropped slots reach nothing; a token whose
    slots are all dropped gets 0; the gradients of dropped rows and weights are 0."""
    ids = np.array([[0, -1], [-1, -1], [1, 0], [-1, 1]])
    _, pos, _ = ref.sort(ids, 2)
    H = 264
    y = torch.full((8, H), 2.0, dtype=TYPES[dtype], device=DEV)
    w = torch.full((4, 2), 0.5, device=DEV)
    for t in range(4):
        for j in range(2):
            if pos[t, j] < 0:
                y[~int(pos[t, j])] = float("nan") if j else float("inf")
                w[t, j] = float("nan")
    pos_t = torch.from_numpy(pos).to(DEV)
    out = b.moe_combine(y, pos_t, w)
    assert torch.equal(out.float().cpu(), torch.tensor([1.0, 0.0, 2.0, 1.0]).unsqueeze(1).expand(4, H))
    back = b.moe_gather_backward(y, pos_t)
    assert torch.equal(back.float().cpu(), torch.tensor([2.0, 0.0, 4.0, 2.0]).unsqueeze(1).expand(4, H))
    d = torch.ones((4, H), dtype=TYPES[dtype], device=DEV)
    d[1] = float("inf")
    d_rows, d_w = b.moe_combine_backward(d, y, pos_t, w)
    assert torch.equal(d_w.cpu(), torch.where(torch.from_numpy(pos) >= 0, 2.0 * H, 0.0))
    want = torch.zeros((8, H))
    for t in range(4):
        for j in range(2):
            if pos[t, j] >= 0:
                want[pos[t, j]] = 0.5
    assert torch.equal(d_rows.float().cpu(), want)
    x = torch.full((4, H), float("nan"), dtype=TYPES[dtype], device=DEV)
    assert torch.equal(torch.isnan(b.moe_gather(x, pos_t)).cpu(), want != 0)


def test_rows_that_lie_apart():
    _, pos, _ = ref.sort(routing(20, 3, 6, seed=1), 6)
    pos_t = torch.from_numpy(pos).to(DEV)
    wide = torch.randn((20, 400), device=DEV)
    for lo, hi in ((0, 256), (1, 258), (4, 24)):             # aligned, misaligned, short rows
        x = wide[:, lo:hi]
        assert torch.equal(b.moe_gather(x, pos_t), b.moe_gather(x.contiguous(), pos_t))
        y = torch.randn((60, hi - lo), device=DEV)
        w = torch.rand((20, 3), device=DEV)
        for g, h in zip(b.moe_combine_backward(x, y, pos_t, w),
                        b.moe_combine_backward(x.contiguous(), y, pos_t, w)):
            # the aligned form may sum d_weights in another order
            assert torch.allclose(g, h, rtol=0, atol=(hi - lo) * 2.0 ** -22)


def test_gradients_against_differences():
    """combine is linear in the rows and in the weights: central differences of the forward pass
    with a step of 1 equal the gradients up to the roundings of the sums."""
    T, top, E, H = 6, 2, 3, 40
    rng = np.random.default_rng(3)
    _, pos, _ = ref.sort(routing(T, top, E, seed=3, drop=0.2), E)
    pos_t = torch.from_numpy(pos).to(DEV)
    y = torch.from_numpy(rng.standard_normal((T * top, H))).float().to(DEV)
    w = torch.from_numpy(rng.random((T, top))).float().to(DEV)
    d = torch.from_numpy(rng.standard_normal((T, H))).float().to(DEV)
    d_rows, d_w = b.moe_combine_backward(d, y, pos_t, w)

    def loss(y, w):
        return (b.moe_combine(y, pos_t, w).double() * d.double()).sum().item()

    tol = T * H * top * 2.0 ** -20
    for t in range(T):
        for j in range(top):
            step = torch.zeros_like(w)
            step[t, j] = 1.0
            assert abs((loss(y, w + step) - loss(y, w - step)) / 2 - d_w[t, j].item()) <= tol
    for r in range(0, T * top, 2):
        step = torch.zeros_like(y)
        step[r, (7 * r) % H] = 1.0
        assert abs((loss(y + step, w) - loss(y - step, w)) / 2 - d_rows[r, (7 * r) % H].item()) <= tol
    x = torch.from_numpy(rng.standard_normal((T, H))).float().to(DEV)
    d_x = b.moe_gather_backward(d_rows, pos_t)

    def spread(x):
        return (b.moe_gather(x, pos_t).double() * d_rows.double()).sum().item()

    for t in range(T):
        step = torch.zeros_like(x)
        step[t, (5 * t) % H] = 1.0
        assert abs((spread(x + step) - spread(x - step)) / 2 - d_x[t, (5 * t) % H].item()) <= tol


# ------------------------------------------------------------------ the experts' products

GROUPS = [(1, 1, 1, 48, 64, 0.0), (1, 4, 32, 272, 544, 0.0), (5, 2, 4, 144, 96, 0.5), (40, 4, 8, 256, 1312, 0.1),
          (64, 2, 130, 80, 288, 0.0), (300, 2, 5, 400, 736, 0.05), (900, 3, 4, 272, 352, 0.0)]


@pytest.mark.parametrize("T,top,E,N,K,drop", GROUPS)
@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_expert_gemm(T, top, E, N, K, drop, gathered, dtype):
    offsets, _, row_token = ref.sort(routing(T, top, E, seed=N, drop=drop, skew=T == 40), E)
    S = T * top
    xq, xs, x = packed(T if gathered else S, K, seed=K)
    ws = [packed(N, K, seed=100 + e, lo=110, hi=130) for e in range(E)]
    out = b.mxfp4_expert_gemm(xq, xs, torch.from_numpy(offsets).to(DEV), torch.stack([w[0] for w in ws]),
                              torch.stack([w[1] for w in ws]),
                              row_token=torch.from_numpy(row_token).to(DEV) if gathered else None,
                              out=torch.full((S, N), 7.0, dtype=TYPES[dtype], device=DEV),
                              out_dtype=TYPES[dtype])
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        if lo < hi:
            check_product(out[lo:hi], x[row_token[lo:hi]] if gathered else x[lo:hi], ws[e][2], dtype)
    assert (out[offsets[E]:] == 0).all()


def check_hidden(hq, hs, h, slack):
    """MXFP4 rows of values known to a relative `slack`: every block's scale is that of a top within
    the slack, every element the rounding of a value within it."""
    q, code = ref.unpack(hq.cpu().numpy(), hs.cpu().numpy())
    m, f = h.shape
    blocks = np.abs(h).reshape(m, f // 32, 32)
    top = blocks.max(axis=2)
    wide = slack.reshape(m, f // 32, 32).max(axis=2)
    low = ref.quantize(np.repeat(np.maximum(top - wide, 0), 32, axis=1))[1]
    high = ref.quantize(np.repeat(top + wide, 32, axis=1))[1]
    assert ((code == low) | (code == high)).all()
    scale = np.ldexp(1.0, np.repeat(code.astype(np.int64), 32, axis=1) - 127)
    got = np.abs(ref.values(q, code)) / scale
    idx = q & 7
    lo = np.where(idx == 0, -1.0, (ref.VALUES[idx] + ref.VALUES[np.maximum(idx, 1) - 1]) / 2)
    hi = np.where(idx == 7, 1e30, (ref.VALUES[idx] + ref.VALUES[np.minimum(idx + 1, 7)]) / 2)
    a, s = np.abs(h) / scale, slack / scale
    assert ((a >= lo - s) & (a <= hi + s)).all()
    assert (np.sign(h) * np.where(q & 8, -1, 1) >= 0)[(got > 0) & (np.abs(h) > slack)].all()
    blocks_stored = code.shape[1]
    pad = hs.cpu().numpy().transpose(1, 0, 2).reshape(m, -1)[:, blocks_stored:]
    assert (pad == 0).all()


@pytest.mark.parametrize("T,top,E,F,K,drop", [(1, 1, 1, 32, 64, 0.0), (1, 4, 32, 288, 544, 0.0),
                                              (40, 4, 8, 256, 1312, 0.1), (300, 2, 5, 736, 352, 0.05),
                                              (900, 3, 4, 160, 288, 0.0)])
@pytest.mark.parametrize("gathered", [False, True])
def test_expert_swiglu(T, top, E, F, K, drop, gathered):
    offsets, _, row_token = ref.sort(routing(T, top, E, seed=F, drop=drop), E)
    S = T * top
    xq, xs, x = packed(T if gathered else S, K, seed=K, lo=122, hi=128)
    ws = [packed(2 * F, K, seed=100 + e, lo=118, hi=124) for e in range(E)]
    hq = torch.full((S, F // 2), 0x77, dtype=torch.uint8, device=DEV)
    hs = torch.full(((F + 255) // 256, S, 8), 0x77, dtype=torch.uint8, device=DEV)
    b.mxfp4_expert_swiglu(xq, xs, torch.from_numpy(offsets).to(DEV), torch.stack([w[0] for w in ws]),
                          torch.stack([w[1] for w in ws]),
                          row_token=torch.from_numpy(row_token).to(DEV) if gathered else None,
                          hq=hq, hs=hs)
    h, slack = np.zeros((S, F)), np.zeros((S, F))
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        xe = x[row_token[lo:hi]] if gathered else x[lo:hi]
        gu, mag = xe @ ws[e][2].T, np.abs(xe) @ np.abs(ws[e][2].T)
        h[lo:hi] = ref.swiglu(gu)
        # errors of gate and up as in check_product; |d silu| <= 1.1, |silu(g)| <= |g|; the
        # activation's own roundings (exp, quotient, product) are below 2^-20 together
        err = mag * (K / 64 + 8) * 2.0 ** -23
        slack[lo:hi] = (1.1 * err[:, 0::2] * np.abs(gu[:, 1::2]) + err[:, 1::2] * np.abs(gu[:, 0::2])
                        + np.abs(h[lo:hi]) * 2.0 ** -20)
    check_hidden(hq, hs, h, slack)
    assert (hq[offsets[E]:] == 0).all() and (hs[:, offsets[E]:] == 0).all()


def test_swiglu_saturated_gates():
    """Gates far below and above zero: the activation goes to 0 and to gate * up without NaN."""
    K, F = 64, 32
    q = np.zeros((2 * F, K), dtype=np.uint8)
    q[0::2, 0] = np.where(np.arange(F) % 2, 7, 15)           # gate +-6, up 1
    q[1::2, 1] = 2
    w = ref.pack(q, np.full((2 * F, 2), 127, dtype=np.uint8))
    xq, code = np.zeros((3, K), dtype=np.uint8), np.full((3, 2), 127, dtype=np.uint8)
    xq[:, 0:2] = 2
    code[1, 0], code[2, 0] = 140, 100                        # gates of 2^13 * 6 and 2^-27 * 6
    x = ref.pack(xq, code)
    offsets = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    hq, hs = b.mxfp4_expert_swiglu(*[torch.from_numpy(t).to(DEV) for t in x], offsets,
                                   torch.from_numpy(w[0][None]).to(DEV), torch.from_numpy(w[1][None]).to(DEV))
    h = ref.swiglu(ref.values(xq, code) @ ref.values(q, np.full((2 * F, 2), 127, dtype=np.uint8)).T)
    check_hidden(hq, hs, h, np.abs(h) * 2.0 ** -20 + 1e-38)


@pytest.mark.parametrize("T,top,E,H,F,dtype,drop", [(1, 2, 4, 256, 96, "bf16", 0.0), (1, 1, 1, 32, 32, "f32", 0.0),
                                                    (3, 2, 5, 288, 160, "f16", 0.3), (2, 3, 8, 1312, 736, "f32", 0.0),
                                                    (1, 4, 16, 4096, 2048, "bf16", 0.0), (8, 8, 16, 256, 96, "bf16", 0.1),
                                                    (70, 2, 6, 288, 160, "f16", 0.1), (600, 4, 4, 512, 288, "f32", 0.0)])
def test_layer_is_its_parts(T, top, E, H, F, dtype, drop):
    """mxfp4_moe is close to the layer in 64 bits; with more slots than the two-launch form takes, it
    gives bit for bit what its parts give (that form sums in another order and does not round the
    experts' outputs)."""
    ids = torch.from_numpy(routing(T, top, E, seed=T, drop=drop)).to(DEV)
    weights = torch.rand((T, top), generator=torch.Generator().manual_seed(1)).to(DEV)
    x, x64 = rows(T, H, dtype, seed=2, spread=0.5)
    w13 = [packed(2 * F, H, seed=10 + e, lo=119, hi=123) for e in range(E)]
    w2 = [packed(H, F, seed=50 + e, lo=119, hi=123) for e in range(E)]
    w13q, w13s = torch.stack([w[0] for w in w13]), torch.stack([w[1] for w in w13])
    w2q, w2s = torch.stack([w[0] for w in w2]), torch.stack([w[1] for w in w2])
    out = b.mxfp4_moe(x, ids, weights, w13q, w13s, w2q, w2s)
    offsets, slot_pos, row_token = b.moe_sort(ids, E)
    xq, xs = b.mxfp4_quantize_rows(x)
    hq, hs = b.mxfp4_expert_swiglu(xq, xs, offsets, w13q, w13s, row_token=row_token)
    y = b.mxfp4_expert_gemm(hq, hs, offsets, w2q, w2s, out_dtype=x.dtype)
    if T * top > 64:
        assert torch.equal(out, b.moe_combine(y, slot_pos, weights))
    off, pos, tok = ref.sort(ids.cpu().numpy(), E)
    xv = ref.values(*ref.quantize(x64))
    y64 = np.zeros((T * top, H))
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        h = ref.swiglu(xv[tok[lo:hi]] @ w13[e][2].T)
        y64[lo:hi] = ref.values(*ref.quantize(h)) @ w2[e][2].T
    want, _ = ref.combine(y64, pos, weights.double().cpu().numpy())
    # hidden elements within the fp32 error (about 2^-17) of a rounding boundary may land on its
    # other side, which moves them by a quarter: a share of 2^-15 of the elements, 2^-9.5 of the
    # norm; the outputs' type adds its own roundings (of y and of out)
    err = np.linalg.norm(out.double().cpu().numpy() - want) / np.linalg.norm(want)
    assert err <= 2.0 ** -8 + 3 * HALF_ULP[dtype]


@pytest.mark.parametrize("T", [2, 50])
def test_layer_dropped_slots(T):
    """Dropped slots add nothing, whatever their weights hold and however their ids are out of range;
    a token without any other slot gets 0."""
    E, H, F = 4, 288, 96
    x, _ = rows(T, H, "bf16", seed=3, spread=0.5)
    w13 = [packed(2 * F, H, seed=10 + e, lo=119, hi=123) for e in range(E)]
    w2 = [packed(H, F, seed=50 + e, lo=119, hi=123) for e in range(E)]
    stacks = [torch.stack([w[i] for w in ws]) for ws in (w13, w2) for i in (0, 1)]
    ids = torch.full((T, 2), 1, dtype=torch.int64, device=DEV)
    ids[0, 1], ids[1] = 2 ** 32 + 1, torch.tensor([-1, E])
    w = torch.full((T, 2), 0.5, device=DEV)
    w[0, 1], w[1] = float("nan"), torch.tensor([float("inf"), float("nan")])
    out = b.mxfp4_moe(x, ids, w, *stacks)
    assert (out[1] == 0).all() and torch.isfinite(out).all()
    one = b.mxfp4_moe(x[:1], ids[:1, :1].contiguous(), w[:1, :1].contiguous(), *stacks)
    # the same sum but for the order of its parts (and the rounding of the experts' outputs)
    assert torch.allclose(out[:1].float(), one.float(), rtol=2.0 ** -6, atol=2.0 ** -8 * one.abs().max().item())
    wide = torch.zeros((T, 400), dtype=torch.bfloat16, device=DEV)
    wide[:, 64:64 + H] = x
    assert torch.equal(b.mxfp4_moe(wide[:, 64:64 + H], ids.to(torch.int32).masked_fill(ids > E, -5), w, *stacks), out)


def test_refusals():
    ids = torch.zeros((4, 2), dtype=torch.int64, device=DEV)
    pos = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV)
    y = torch.zeros((8, 64), dtype=torch.bfloat16, device=DEV)
    w = torch.zeros((4, 2), device=DEV)
    with pytest.raises(TypeError):
        b.moe_sort(ids.float(), 4)
    with pytest.raises(b.W8A8Error):
        b.moe_sort(ids, 0)
    with pytest.raises(b.W8A8Error):
        b.moe_sort(ids, b.MOE_MAX_EXPERTS + 1)
    with pytest.raises(ValueError):
        b.moe_gather(x[:3], pos)
    with pytest.raises(TypeError):
        b.moe_gather(x, pos.long())
    with pytest.raises(ValueError):
        b.moe_combine(y[:7], pos, w)
    with pytest.raises(TypeError):
        b.moe_combine(y, pos, w.to(torch.bfloat16))
    with pytest.raises(ValueError):
        b.moe_combine_backward(x.float(), y, pos, w)
    wq, ws, _ = packed(64, 64, seed=1)
    offsets = torch.tensor([0, 8], dtype=torch.int32, device=DEV)
    yq, ys = b.mxfp4_quantize_rows(y)
    with pytest.raises(ValueError):
        b.mxfp4_expert_gemm(yq, ys, offsets[:1], wq[None], ws[None])
    with pytest.raises(ValueError):
        b.mxfp4_expert_swiglu(yq, ys, offsets, wq[None, :48].contiguous(), ws[None, :, :48].contiguous())
    with pytest.raises(ValueError):
        b.mxfp4_moe(x, ids, w, wq[None], ws[None], wq[None], ws[None])   # w2 is not [H, F]


@pytest.mark.parametrize("T,top,E,H,F", [(1, 1, 2, 64, 2080), (1, 3, 4, 96, 800), (2, 4, 6, 160, 544), (1, 5, 8, 320, 1056),
                                         (1, 8, 8, 1056, 2080), (8, 1, 3, 32, 1312), (4, 2, 5, 2080, 288)])
@pytest.mark.parametrize("drop", [0.0, 0.4])
def test_few_slots_of_every_depth(T, top, E, H, F, drop):
    """The layer of a few slots with one to nine items of K per wavefront and more, slots without an
    expert between them: as in 64 bits (bound as above), and the same bits in every run."""
    ids = torch.from_numpy(routing(T, top, E, seed=H + T, drop=drop)).to(DEV)
    weights = torch.rand((T, top), generator=torch.Generator().manual_seed(1)).to(DEV)
    x, x64 = rows(T, H, "f32", seed=2, spread=0.5)
    w13 = [packed(2 * F, H, seed=10 + e, lo=119, hi=123) for e in range(E)]
    w2 = [packed(H, F, seed=50 + e, lo=119, hi=123) for e in range(E)]
    stacks = [torch.stack([w[i] for w in ws]) for ws in (w13, w2) for i in (0, 1)]
    runs = [b.mxfp4_moe(x, ids, weights, *stacks) for _ in range(20)]
    assert all(torch.equal(runs[0], r) for r in runs[1:])
    xv = ref.values(*ref.quantize(x64))
    want = np.zeros((T, H))
    for t, slots in enumerate(ids.tolist()):
        for j, e in enumerate(slots):
            if e >= 0:
                h = ref.values(*ref.quantize(ref.swiglu(xv[t:t + 1] @ w13[e][2].T)))
                want[t] += weights[t, j].item() * (h @ w2[e][2].T)[0]
    err = np.linalg.norm(runs[0].double().cpu().numpy() - want)
    assert err <= (2.0 ** -8 + 3 * HALF_ULP["f32"]) * np.linalg.norm(want)
