"""MXFP4 rows and products on the GPU against their definitions in 64 bits."""
import numpy as np
import pytest
import torch

import mx_reference as ref
from quantized_gemm_quantize_amd import binding as b

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# half a unit in the last place, relative (eps is the step above 1)
HALF_ULP = {d: torch.finfo(t).eps / 2 for d, t in TYPES.items()}
# smallest step of the type (below its normal range)
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24, "f32": 2.0 ** -149}


def rows(m, k, dtype, seed, spread=3.0):
    """Rows whose blocks have magnitudes spread over 2^(+-3 spread)."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, k)) * np.exp2(np.repeat(rng.standard_normal((m, k // 32)) * spread, 32, axis=1))
    t = torch.from_numpy(x).to(TYPES[dtype])
    return t.to(DEV), t.double().numpy()


def packed(m, k, seed, lo=100, hi=140):
    """Random MXFP4 storage: (codes, scales) on the GPU and their values in 64 bits."""
    rng = np.random.default_rng(seed)
    q = rng.integers(0, 16, (m, k)).astype(np.uint8)
    code = rng.integers(lo, hi, (m, k // 32)).astype(np.uint8)
    c, s = ref.pack(q, code)
    return torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV), ref.values(q, code)


def check_product(got, x, w, dtype):
    """The products are exact; each of the K / 64 accumulations of a chain, and the at most 8
    joins of partial sums, rounds to 2^-23 of the partial sum's size at worst; the result rounds
    to its type once."""
    want = x @ w.T
    mag = np.abs(x) @ np.abs(w.T)
    steps = x.shape[1] / 64 + 8
    bound = mag * steps * 2.0 ** -23 + np.abs(want) * HALF_ULP[dtype] * 1.001 + TINY[dtype]
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= bound).all(), f"worst {np.max(err / bound)} of the bound"


# ------------------------------------------------------------------ rows

@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,k", [(1, 32), (1, 4096), (3, 96), (7, 256), (33, 288), (130, 736), (257, 1312), (64, 8192)])
def test_quantize_is_exact(dtype, m, k):
    x, x64 = rows(m, k, dtype, seed=m * 1000 + k)
    codes, scales = b.mxfp4_quantize_rows(x)
    c, s = ref.pack(*ref.quantize(x64))
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), c)
    back = b.mxfp4_dequantize_rows(codes, scales, TYPES[dtype])
    want = torch.from_numpy(ref.values(*ref.quantize(x64))).to(TYPES[dtype])
    assert torch.equal(back.cpu(), want)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quantize_special_blocks(dtype):
    """Zeros, negative zeros, ties of every grid step, saturation (top in (6, 8) steps),
    subnormals, the largest finite value, and every power of two as the largest magnitude."""
    info = torch.finfo(TYPES[dtype])
    blocks = [np.zeros(32), -np.zeros(32)]
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 1, 1.5, 2, 3, 4, 6, 7, 7.75])
    for e in (-10, 0, 7):
        blocks.append(np.ldexp(np.concatenate([ties, -ties]), e))
    tiny = float(info.smallest_normal) * float(info.eps)
    blocks.append(tiny * np.arange(32))
    blocks.append(np.where(np.arange(32) == 5, float(info.max), 1.0))
    lo, hi = (-149, 127) if dtype == "f32" else (-133, 127) if dtype == "bf16" else (-24, 15)
    for e in range(lo, hi + 1):
        blocks.append(np.ldexp(np.linspace(-1.0, 1.0, 32).round(2), e))
    x = torch.from_numpy(np.stack(blocks)).to(TYPES[dtype])
    codes, scales = b.mxfp4_quantize_rows(x.to(DEV))
    c, s = ref.pack(*ref.quantize(x.double().numpy()))
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), c)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quantize_non_finite_blocks_are_nan(dtype):
    x, _ = rows(4, 320, dtype, seed=5)
    x[0, 33], x[1, 0], x[2, 319] = float("nan"), float("inf"), float("-inf")
    codes, scales = b.mxfp4_quantize_rows(x)
    c, s = ref.pack(*ref.quantize(x.double().cpu().numpy()))
    assert np.array_equal(scales.cpu().numpy(), s) and np.array_equal(codes.cpu().numpy(), c)
    nan = torch.isnan(b.mxfp4_dequantize_rows(codes, scales, TYPES[dtype])).cpu().numpy()
    want = np.zeros((4, 320), dtype=bool)
    want[0, 32:64], want[1, 0:32], want[2, 288:320] = True, True, True
    assert np.array_equal(nan, want)


def test_quantize_rows_that_lie_apart():
    base, _ = rows(9, 512, "bf16", seed=6)
    x = base[:, 64:64 + 288]
    codes, scales = b.mxfp4_quantize_rows(x)
    same = b.mxfp4_quantize_rows(x.contiguous())
    assert torch.equal(codes, same[0]) and torch.equal(scales, same[1])
    one = b.mxfp4_quantize_rows(base[3:4, 64:64 + 288])
    assert torch.equal(one[0][0], codes[3])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_dequantize_every_code(dtype):
    """All 16 elements at every scale code, the overflow and NaN ones included."""
    q = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    code = np.arange(256, dtype=np.uint8).reshape(256, 1)
    c, s = ref.pack(q, code)
    got = b.mxfp4_dequantize_rows(torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV), TYPES[dtype])
    want = torch.from_numpy(ref.values(q, code)).to(torch.float32).to(TYPES[dtype])
    assert torch.equal(got.cpu().nan_to_num(nan=123.0), want.nan_to_num(nan=123.0))


# ------------------------------------------------------------------ the product

SHAPES = [(1, 16, 32), (1, 4096, 4096), (2, 48, 64), (5, 272, 96), (16, 256, 256), (17, 144, 288),
          (31, 1040, 736), (33, 512, 1312), (64, 1024, 2048), (65, 80, 4096), (129, 640, 160),
          (200, 208, 544), (257, 1040, 1312), (300, 400, 5120), (513, 272, 1024)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_gemm(m, n, k, dtype):
    xq, xs, x = packed(m, k, seed=m + n)
    wq, ws, w = packed(n, k, seed=k, lo=105 if dtype != "f16" else 118, hi=130 if dtype != "f16" else 128)
    if dtype == "f16":                       # keep the sums inside binary16
        xq, xs, x = packed(m, k, seed=m + n, lo=115, hi=126)
    check_product(b.mxfp4_gemm(xq, xs, wq, ws, out_dtype=TYPES[dtype]), x, w, dtype)


def test_gemm_large_tiles():
    """Enough rows and columns for the largest tiles, ragged in both."""
    xq, xs, x = packed(4100, 512, seed=1)
    wq, ws, w = packed(4112, 512, seed=2)
    check_product(b.mxfp4_gemm(xq, xs, wq, ws, out_dtype=torch.float32), x, w, "f32")


def test_gemm_asks_for_every_block():
    """A single nonzero element in every position of K in turn: each block meets its own scale."""
    k = 544
    q = np.zeros((k, k), dtype=np.uint8)
    np.fill_diagonal(q, 2)                                  # 1.0
    code = np.broadcast_to(110 + np.arange(k // 32, dtype=np.uint8), (k, k // 32)).copy()
    c, s = ref.pack(q, code)
    xq, xs = torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV)
    wq, ws, w = packed(48, k, seed=3)
    got = b.mxfp4_gemm(xq, xs, wq, ws, out_dtype=torch.float32).double().cpu().numpy()
    assert np.array_equal(got, ref.values(q, code) @ w.T)   # one term each: exact


@pytest.mark.parametrize("m", [3, 40, 300])
def test_gemm_nan_rows(m):
    """A NaN block of x makes its row NaN, one of w its column, and nothing else."""
    xq, xs, x = packed(m, 288, seed=4)
    wq, ws, w = packed(80, 288, seed=5)
    xs[1, 2, 0] = 255
    ws[0, 33, 7] = 255
    out = b.mxfp4_gemm(xq, xs, wq, ws, out_dtype=torch.float32).cpu()
    nan = torch.zeros((m, 80), dtype=torch.bool)
    nan[2, :], nan[:, 33] = True, True
    assert torch.equal(torch.isnan(out), nan)


@pytest.mark.parametrize("x_dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1, 512, 4096), (3, 48, 32), (4, 272, 1312), (5, 1040, 96), (1, 8208, 96),
                                   (37, 272, 352), (300, 640, 1312)])
def test_linear(m, n, k, x_dtype):
    x, x64 = rows(m, k, x_dtype, seed=m, spread=1.0)
    wq, ws, w = packed(n, k, seed=n, lo=112, hi=120)
    got = b.mxfp4_linear(x, wq, ws, out_dtype=torch.float32)
    check_product(got, ref.values(*ref.quantize(x64)), w, "f32")
    assert torch.equal(b.mxfp4_linear(x, wq, ws), got.to(TYPES[x_dtype]))
    work = torch.empty(b.mxfp4_linear_workspace(m, n, k), dtype=torch.uint8, device=DEV)
    assert torch.equal(b.mxfp4_linear(x, wq, ws, out_dtype=torch.float32, workspace=work), got)


@pytest.mark.parametrize("m", [2, 40])
def test_linear_non_finite_and_apart(m):
    """A row with an infinity or NaN gives a NaN row and leaves the others; rows may lie apart."""
    base, _ = rows(m, 512, "bf16", seed=8)
    x = base[:, 64:64 + 352]
    x[1, 40] = float("nan")
    wq, ws, _ = packed(64, 352, seed=9)
    out = b.mxfp4_linear(x, wq, ws)
    assert torch.isnan(out[1]).all() and torch.isfinite(out[:1]).all() and torch.isfinite(out[2:]).all()
    assert torch.equal(out.nan_to_num(), b.mxfp4_linear(x.contiguous(), wq, ws).nan_to_num())


def test_empty():
    wq, ws, _ = packed(32, 64, seed=1)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    codes, scales = b.mxfp4_quantize_rows(x)
    assert codes.shape == (0, 32) and scales.shape == (1, 0, 8)
    assert b.mxfp4_dequantize_rows(codes, scales).shape == (0, 64)
    assert b.mxfp4_gemm(codes, scales, wq, ws).shape == (0, 32)
    assert b.mxfp4_linear(x, wq, ws).shape == (0, 32)


def test_refusals():
    wq, ws, _ = packed(32, 64, seed=1)
    x, _ = rows(4, 64, "bf16", seed=1)
    with pytest.raises(TypeError):
        b.mxfp4_quantize_rows(x.double())
    with pytest.raises(ValueError):
        b.mxfp4_quantize_rows(x.cpu())
    with pytest.raises(ValueError):
        b.mxfp4_quantize_rows(x.t())                         # rows are not contiguous
    with pytest.raises(b.W8A8Error):
        b.mxfp4_quantize_rows(x[:, :40])                     # K is not a multiple of 32
    with pytest.raises(b.W8A8Error):
        b.mxfp4_quantize_rows(x[:, 1:33])                    # misaligned rows
    with pytest.raises(b.W8A8Error):
        b.mxfp4_quantize_rows(x[:1].expand(4, 64))           # rows on top of each other
    with pytest.raises(ValueError):
        b.mxfp4_gemm(wq, ws[:, :16], wq, ws)                 # scales of other rows
    with pytest.raises(ValueError):
        b.mxfp4_gemm(wq[:, :16].contiguous(), ws, wq, ws)    # another K
    with pytest.raises(b.W8A8Error):
        b.mxfp4_gemm(wq, ws, wq[:24].contiguous(), ws[:, :24].contiguous())  # N not a multiple of 16
    with pytest.raises(TypeError):
        b.mxfp4_gemm(wq, ws, wq, ws, out_dtype=torch.float64)
    with pytest.raises(b.W8A8Error):
        b.mxfp4_linear(rows(12, 64, "bf16", seed=1)[0], wq, ws,
                       workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
