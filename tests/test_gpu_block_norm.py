"""Block norms and their gradients on the GPU against their definitions in 64 bits."""
import numpy as np
import pytest
import torch

import block_reference as ref
from quantized_gemm_quantize_amd import binding as b

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-5
# one element, one thread's chunk and its neighbours, wavefronts, workgroups, the widest rows, odd widths
WIDTHS = [1, 7, 8, 9, 64, 257, 512, 513, 1031, 1280, 2056, 4096, 5120, 8200, 16384]


def case(T, H, dtype, seed, gate="none", post=False):
    rng = np.random.default_rng(seed)
    v = {}
    for name in ("r", "y", "d_out", "d_new"):
        x = rng.standard_normal((T, H)) * (3.0 if name == "r" else 1.0)
        if T > 2:
            x[2] = 0.0      # a row of zeros: eps alone under the root
        v[name], v[name + "64"] = ref.rounded(x, dtype)
        v[name] = v[name].to(DEV)
    for name in ("weight", "post_weight"):
        v[name], v[name + "64"] = ref.rounded(1 + 0.3 * rng.standard_normal(H), "f32")
        v[name] = v[name].to(DEV)
    if not post:
        v["post_weight"] = v["post_weight64"] = None
    v["gate"] = v["gate64"] = None
    if gate != "none":
        g = rng.standard_normal(H if gate == "channel" else (T, H))
        v["gate"], v["gate64"] = ref.rounded(g, "f32" if gate == "channel" else dtype)
        v["gate"] = v["gate"].to(DEV)
    return v


def forward_want(v, post, scale=0.7):
    return ref.block_norm(v["r64"], v["y64"], post, v["post_weight64"], v["gate64"], scale, v["weight64"], EPS)


def forward_args(v, post, scale=0.7):
    return dict(y=v["y"], post_norm=post, post_weight=v["post_weight"], gate=v["gate"], scale=scale, eps=EPS)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("H", WIDTHS)
def test_forward_widths(dtype, H):
    for T, gate, post in ((1, "none", False), (5, "channel", True), (11, "token", True)):
        v = case(T, H, dtype, seed=H, gate=gate, post=post)
        new, e_new, out, e_out = forward_want(v, post)
        got_new, got = b.block_norm(v["r"], v["weight"], **forward_args(v, post))
        ref.close(got_new, new, e_new, dtype, f"residual {T} {gate}")
        ref.close(got, out, e_out, dtype, f"out {T} {gate}")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("H", WIDTHS)
def test_plain_norm(dtype, H):
    v = case(4, H, dtype, seed=2)
    new, out = b.block_norm(v["r"], v["weight"], eps=EPS)
    assert new is v["r"]
    _, _, want, e = ref.block_norm(v["r64"], weight=v["weight64"], eps=EPS)
    ref.close(out, want, e, dtype)
    _, ones = b.block_norm(v["r"], eps=EPS)
    _, _, want, e = ref.block_norm(v["r64"], eps=EPS)
    ref.close(ones, want, e, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("post", [False, True])
def test_many_rows(dtype, post):
    v = case(4099, 264, dtype, seed=3, gate="token", post=post)
    new, e_new, out, e_out = forward_want(v, post)
    got_new, got = b.block_norm(v["r"], v["weight"], **forward_args(v, post))
    ref.close(got_new, new, e_new, dtype)
    ref.close(got, out, e_out, dtype)


def apart(t, extra, offset=0):
    """The same rows with a stride of width + extra elements, `offset` elements into the buffer; the gaps
    hold NaN."""
    T, H = t.shape
    flat = torch.full((T * (H + extra) + offset,), float("nan"), dtype=t.dtype, device=t.device)
    rows = flat[offset:].view(T, H + extra)[:, :H]
    rows.copy_(t)
    return rows


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("extra,offset", [(8, 0), (1, 0), (3, 1), (5, 7)])
@pytest.mark.parametrize("H", [264, 1031])
def test_rows_apart_and_unaligned(dtype, extra, offset, H):
    v = case(6, H, dtype, seed=4, gate="token", post=True)
    new, e_new, out, e_out = forward_want(v, True)
    args = forward_args(v, True)
    args.update(y=apart(v["y"], extra, offset), gate=apart(v["gate"], extra + 2, offset))
    got_new, got = b.block_norm(apart(v["r"], extra, offset), v["weight"], **args)
    ref.close(got_new, new, e_new, dtype)
    ref.close(got, out, e_out, dtype)
    # gradients, and outputs at unaligned addresses
    r, r64 = ref.rounded(new, dtype)
    want = ref.block_norm_backward(v["d_out64"], v["d_new64"], r64, v["y64"], True, v["post_weight64"], v["gate64"], 0.7,
                                   v["weight64"], EPS)
    found = b.block_norm_backward(apart(v["d_out"], extra, offset), apart(r.to(DEV), extra, offset), v["weight"],
                                  d_residual=apart(v["d_new"], extra, offset), **args)
    check_gradients(found, want, dtype)
    flat = torch.full((6 * H + 9,), 7.0, dtype=ref.TYPES[dtype], device=DEV)
    b.block_norm(v["r"], v["weight"], out=flat[3:3 + 6 * H].view(6, H), **forward_args(v, True))
    assert torch.equal(flat[3:3 + 6 * H].view(6, H), got)
    assert (flat[:3] == 7).all() and (flat[3 + 6 * H:] == 7).all()


def check_gradients(found, want, dtype):
    found = dict(zip(("d_residual", "d_weight", "d_y", "d_post_weight", "d_gate"), found))
    for name, t in found.items():
        if name not in want:
            assert t is None, name
            continue
        value, bound = want[name]
        ref.close(t, value, bound, dtype if t.dim() == 2 else "f32", name)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("H", WIDTHS)
def test_backward_widths(dtype, H):
    for T, gate, post in ((1, "token", False), (5, "channel", True), (12, "token", True), (3, "none", True)):
        v = case(T, H, dtype, seed=H + 1, gate=gate, post=post)
        want = ref.block_norm_backward(v["d_out64"], v["d_new64"], v["r64"], v["y64"], post, v["post_weight64"],
                                       v["gate64"], 0.7, v["weight64"], EPS)
        found = b.block_norm_backward(v["d_out"], v["r"], v["weight"], d_residual=v["d_new"], **forward_args(v, post))
        check_gradients(found, want, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(4099, 264), (2500, 1031), (1300, 4104)])
def test_backward_many_rows(dtype, T, H):
    v = case(T, H, dtype, seed=5, gate="channel", post=True)
    want = ref.block_norm_backward(v["d_out64"], v["d_new64"], v["r64"], v["y64"], True, v["post_weight64"], v["gate64"],
                                   0.7, v["weight64"], EPS)
    found = b.block_norm_backward(v["d_out"], v["r"], v["weight"], d_residual=v["d_new"], **forward_args(v, True))
    check_gradients(found, want, dtype)
    again = b.block_norm_backward(v["d_out"], v["r"], v["weight"], d_residual=v["d_new"], **forward_args(v, True))
    assert all(torch.equal(x, y) for x, y in zip(found, again))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_without_a_block_output(dtype):
    v = case(9, 520, dtype, seed=6)
    for d_new in (None, v["d_new"]):
        want = ref.block_norm_backward(v["d_out64"], 0.0 if d_new is None else v["d_new64"], v["r64"],
                                       weight=v["weight64"], eps=EPS)
        found = b.block_norm_backward(v["d_out"], v["r"], v["weight"], d_residual=d_new, eps=EPS)
        check_gradients(found, want, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,H", [(1, 16), (3, 48), (5, 512), (7, 1040), (4, 4096), (3, 5120), (2, 16384), (2050, 272)])
def test_int8_rows(dtype, T, H):
    v = case(T, H, dtype, seed=7, gate="channel", post=True)
    new, e_new, out, e = forward_want(v, True)
    got_new, xq, xs = b.block_norm_w8a8(v["r"], v["weight"], **forward_args(v, True))
    ref.close(got_new, new, e_new, dtype)
    xs, xq = xs.double().cpu().numpy(), xq.cpu().numpy().astype(np.float64)
    s = np.abs(out).max(axis=1) / 127
    e_s = e.max(axis=1) / 127 + 2 * ref.U * s
    assert (np.abs(xs - s) <= e_s).all()
    # codes: half a step, and what the row and its scale may be off by, in steps
    s, e_s = np.maximum(s, 1e-300)[:, None], e_s[:, None]
    limit = 0.5 + e / s + 127 * e_s / s + 1e-5
    assert (np.abs(xq - out / s) <= limit).all() and np.abs(xq).max() <= 127
    assert (np.abs(xq).max(axis=1) == np.where(xs > 0, 127, 0)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,H", [(1, 32), (3, 96), (5, 512), (7, 1056), (4, 4096), (3, 5120), (2, 16384), (2050, 288)])
def test_mxfp4_rows(dtype, T, H):
    v = case(T, H, dtype, seed=8, gate="token", post=True)
    new, e_new, out, e = forward_want(v, True)
    got_new, codes, scales = b.block_norm_mxfp4(v["r"], v["weight"], **forward_args(v, True))
    ref.close(got_new, new, e_new, dtype)
    blocks = H // 32
    code = scales.permute(1, 0, 2).reshape(T, -1).cpu().numpy().astype(np.int64)
    assert (code[:, blocks:] == 0).all()
    code = code[:, :blocks]
    o, e = out.reshape(T, blocks, 32), e.reshape(T, blocks, 32)
    top, slack = np.abs(o).max(axis=2), e.max(axis=2)

    def scale_code(a):
        return np.where(a > 0, np.maximum(np.floor(np.log2(np.maximum(a, 1e-300))) - 2, -127) + 127, 0)

    assert (code >= scale_code(top - slack)).all() and (code <= scale_code(top + slack)).all()
    step = np.exp2(code - 127.0)[..., None]
    got = b.mxfp4_dequantize_rows(codes, scales, torch.float32).double().cpu().numpy().reshape(o.shape)

    def grid(a):
        """To the nearest element, ties to even."""
        a = np.clip(a / step, -8, 8)
        s = np.exp2(np.clip(np.floor(np.log2(np.maximum(np.abs(a), 1e-300))), 0, 2) - 1)
        return np.clip(np.round(a / s) * s, -6, 6) * step

    assert (got >= grid(o - e)).all() and (got <= grid(o + e)).all()


def test_quantized_rows_are_those_of_the_quantizers():
    """Without y or weights the output is exact in binary32 for rows of +-1: int8 and MXFP4 rows are then what
    the row quantizations make of it."""
    g = torch.Generator(device=DEV).manual_seed(1)
    x = (torch.randint(0, 2, (33, 512), generator=g, device=DEV) * 2 - 1).to(torch.bfloat16)
    w = torch.randint(-1000, 1000, (512,), generator=g, device=DEV).float() / 64
    _, out = b.block_norm(x.float(), w, eps=1e-30)
    _, xq, xs = b.block_norm_w8a8(x, w, eps=1e-30)
    q, s = b.w8a8_quantize_rows_f32(out)
    assert torch.equal(xq, q) and torch.equal(xs, s)
    _, codes, scales = b.block_norm_mxfp4(x, w, eps=1e-30)
    c, sc = b.mxfp4_quantize_rows(out)
    assert torch.equal(codes, c) and torch.equal(scales, sc)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(dtype):
    v = case(70, 1032, dtype, seed=9, gate="token", post=True)
    want_new, want = b.block_norm(v["r"], v["weight"], **forward_args(v, True))
    for target in ("r", "y"):
        c = {k: t.clone() if isinstance(t, torch.Tensor) else t for k, t in v.items()}
        new, out = b.block_norm(c["r"], c["weight"], new_residual=c[target], **forward_args(c, True))
        assert new is c[target] and torch.equal(new, want_new) and torch.equal(out, want)


def test_no_rows_and_not_finite():
    empty = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    gate = torch.ones(64, device=DEV)
    new, out = b.block_norm(empty, y=empty, gate=gate)
    assert new.shape == out.shape == (0, 64)
    found = b.block_norm_backward(empty, empty, y=empty, gate=gate, post_norm=True)
    torch.cuda.synchronize()
    assert all((found[i] == 0).all() and found[i].shape == (64,) for i in (1, 3, 4))
    # a NaN and an infinity stay in their rows
    x = torch.ones((4, 256), dtype=torch.float32, device=DEV)
    x[1, 5], x[2, 7] = float("nan"), float("inf")
    _, out = b.block_norm(x, eps=EPS)
    assert out[0].isfinite().all() and out[3].isfinite().all()
    assert out[1].isnan().all() and out[2, 7].isnan() and (out[2, :7] == 0).all()
    _, codes, scales = b.block_norm_mxfp4(x, eps=EPS)
    back = b.mxfp4_dequantize_rows(codes, scales, torch.float32)
    assert back[1].isnan().all() and back[2, :32].isnan().all() and (back[2, 32:] == 0).all()
    assert back[0].isfinite().all() and back[3].isfinite().all()


def test_rows_behind_the_last_are_left():
    buffer = torch.full((9, 136), 5.0, dtype=torch.bfloat16, device=DEV)
    x = torch.randn((4, 136), device=DEV).to(torch.bfloat16)
    b.block_norm(x, out=buffer[:4])
    assert (buffer[4:] == 5).all()


def test_offsets_beyond_32_bits():
    """Rows that lie more than 2^31 elements apart in all."""
    T, H, ld = 5, 264, 2 ** 29 + 8
    buffer = torch.empty((T - 1) * ld + H, dtype=torch.bfloat16, device=DEV)
    rows = torch.as_strided(buffer, (T, H), (ld, 1))
    v = case(T, H, "bf16", seed=10)
    rows.copy_(v["r"])
    _, out = b.block_norm(rows, v["weight"], eps=EPS)
    _, want = b.block_norm(v["r"], v["weight"], eps=EPS)
    assert torch.equal(out, want)


def test_expanded_rows_are_refused():
    x = torch.ones((4, 64), dtype=torch.bfloat16, device=DEV)
    one = torch.ones((1, 64), dtype=torch.bfloat16, device=DEV).expand(4, 64)
    for kw in (dict(gate=one), dict(y=one)):
        with pytest.raises(ValueError):
            b.block_norm(x, **{"y": x, **kw})
        with pytest.raises(ValueError):
            b.block_norm_backward(x, x, **{"y": x, **kw})
    with pytest.raises(b.W8A8Error):
        b.block_norm(one)
    with pytest.raises(ValueError):
        b.w16a16_linear(x, torch.ones((64, 64), dtype=torch.bfloat16, device=DEV), residual=one)
