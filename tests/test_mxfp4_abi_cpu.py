"""Refusals of the MXFP4 and expert entry points, without a GPU: every invalid argument gets its
documented status before any HIP call (pointers here are never dereferenced)."""
import os
import re

import pytest

from quantized_gemm_quantize_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "w8a8.h")
OK, NULL, SHAPE, ALIGN, DTYPE = 0, -1, -2, -3, -6
P = 0x10000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("libw8a8.so not built")
    return binding.load()


def test_library_exports_every_declared_symbol(lib):
    names = set(re.findall(r"^[\w ]*\b((?:mxfp4|moe)_\w+)\s*\(", open(HEADER).read(), re.M))
    assert len(names) == 15
    for fn in names:
        assert hasattr(lib, fn), fn


def test_header_constants_match_binding():
    text = open(HEADER).read()
    assert f"#define MXFP4_MAX_K {binding.MXFP4_MAX_K}" in text
    assert f"#define MOE_MAX_EXPERTS {binding.MOE_MAX_EXPERTS}" in text
    for name in ("MXFP4_BF16", "MXFP4_F16", "MXFP4_F32"):
        assert re.search(rf"{name}\s*=\s*{getattr(binding, name)}\b", text)


def caller(f, order, base):
    """f with named arguments over a valid call."""
    def call(**kw):
        assert set(kw) <= set(order)
        return f(*[kw.get(n, base[n]) for n in order])
    return call


QUANT = dict(x=P, ldx=64, M=4, K=64, dt=0, codes=P, scales=P, stream=None)
GEMM = dict(xq=P, xs=P, M=4, wq=P, ws=P, N=32, K=64, dt=0, out=P, stream=None)


def test_quantize(lib):
    c = caller(lib.mxfp4_quantize_rows, list(QUANT), QUANT)
    assert c(M=-1) == SHAPE and c(K=0) == SHAPE and c(K=48, ldx=48) == SHAPE
    assert c(K=binding.MXFP4_MAX_K + 32, ldx=2 ** 21) == SHAPE
    assert c(ldx=32) == SHAPE and c(ldx=2 ** 31) == SHAPE and c(M=2 ** 27) == SHAPE and c(M=2 ** 40) == SHAPE
    assert c(dt=3) == DTYPE and c(dt=-1) == DTYPE
    for n in ("x", "codes", "scales"):
        assert c(**{n: 0}) == NULL and c(**{n: P + 8}) == ALIGN
    assert c(ldx=68) == ALIGN and c(ldx=66, dt=2) == ALIGN
    assert c(M=0, x=0, codes=0, scales=0) == OK


def test_dequantize(lib):
    base = dict(codes=P, scales=P, M=4, K=64, dt=0, out=P, stream=None)
    c = caller(lib.mxfp4_dequantize_rows, list(base), base)
    assert c(M=-1) == SHAPE and c(K=40) == SHAPE and c(dt=9) == DTYPE
    for n in ("codes", "scales", "out"):
        assert c(**{n: 0}) == NULL and c(**{n: P + 4}) == ALIGN
    assert c(M=0, codes=0, scales=0, out=0) == OK


def test_gemm(lib):
    c = caller(lib.mxfp4_gemm, list(GEMM), GEMM)
    assert c(M=-1) == SHAPE and c(N=0) == SHAPE and c(N=24) == SHAPE and c(K=16) == SHAPE
    assert c(N=2 ** 28) == SHAPE and c(dt=3) == DTYPE
    for n in ("xq", "xs", "wq", "ws", "out"):
        assert c(**{n: 0}) == NULL and c(**{n: P + 2}) == ALIGN
    assert c(M=0, xq=0, xs=0, out=0) == OK


def test_linear(lib):
    base = dict(x=P, ldx=64, xd=0, M=40, wq=P, ws=P, N=32, K=64, od=0, out=P, work=P, size=1 << 20, stream=None)
    c = caller(lib.mxfp4_linear, list(base), base)
    need = lib.mxfp4_linear_workspace(40, 32, 64)
    assert need >= 40 * 32 + 40 * 8 and lib.mxfp4_linear_workspace(0, 32, 64) == 0
    assert lib.mxfp4_linear_workspace(40, 32, 60) == 0
    # a few rows: no workspace, one may be given all the same
    assert lib.mxfp4_linear_workspace(4, 32, 64) == 0 and lib.mxfp4_linear_workspace(5, 32, 64) > 0
    assert lib.mxfp4_linear_workspace(1, 8208, 64) > 0
    assert c(M=4, work=0, size=0, out=0) == NULL and c(M=5, size=0) == SHAPE and c(M=4, work=P + 8) == ALIGN
    assert c(size=need - 1) == SHAPE and c(M=-1) == SHAPE and c(N=8) == SHAPE and c(ldx=63) == SHAPE
    assert c(xd=4) == DTYPE and c(od=-2) == DTYPE
    for n in ("x", "wq", "ws", "out", "work"):
        assert c(**{n: 0}) == NULL and c(**{n: P + 8}) == ALIGN
    assert c(ldx=68) == ALIGN
    assert c(M=0, x=0, out=0, work=0, size=0) == OK


def test_sort(lib):
    base = dict(ids=P, bits=32, T=4, top=2, E=8, offsets=P, pos=P, tok=P, work=0, size=0, stream=None)
    c = caller(lib.moe_sort, list(base), base)
    assert c(T=-1) == SHAPE and c(top=0) == SHAPE and c(E=0) == SHAPE and c(E=513) == SHAPE
    assert c(T=2 ** 24) == SHAPE and c(T=2 ** 20, top=2 ** 10) == SHAPE
    assert c(bits=16) == DTYPE
    need = lib.moe_sort_workspace(100000, 8)
    assert need > 0 and c(T=50000, size=need - 4) == SHAPE and c(T=50000, size=need) == NULL
    for n in ("ids", "offsets", "pos", "tok"):
        assert c(**{n: 0}) == NULL and c(**{n: P + 2}) == ALIGN
    assert c(ids=P + 4, bits=64) == ALIGN


def test_rows(lib):
    g = dict(x=P, ldx=8, pos=P, T=4, top=2, H=8, dt=0, rows=P, stream=None)
    c = caller(lib.moe_gather, list(g), g)
    assert c(T=-1) == SHAPE and c(H=0) == SHAPE and c(ldx=7) == SHAPE and c(H=2 ** 24, ldx=2 ** 24) == SHAPE
    assert c(dt=3) == DTYPE and c(x=0) == NULL and c(pos=0) == NULL and c(rows=0) == NULL
    assert c(x=P + 1) == ALIGN and c(x=P + 2, dt=2) == ALIGN and c(pos=P + 2) == ALIGN and c(rows=P + 1) == ALIGN
    assert c(T=0, x=0, pos=0, rows=0) == OK
    g = dict(rows=P, pos=P, T=4, top=2, H=8, dt=0, out=P, stream=None)
    c = caller(lib.moe_gather_backward, list(g), g)
    assert c(top=0) == SHAPE and c(dt=-1) == DTYPE and c(rows=0) == NULL and c(out=P + 1) == ALIGN
    g = dict(rows=P, pos=P, w=P, T=4, top=2, H=8, dt=0, out=P, stream=None)
    c = caller(lib.moe_combine, list(g), g)
    assert c(top=0) == SHAPE and c(dt=-1) == DTYPE and c(w=0) == NULL and c(w=P + 2) == ALIGN
    assert c(T=0, rows=0, pos=0, w=0, out=0) == OK
    g = dict(d=P, ldd=8, rows=P, pos=P, w=P, T=4, top=2, H=8, dt=0, dr=P, dw=P, stream=None)
    c = caller(lib.moe_combine_backward, list(g), g)
    assert c(ldd=7) == SHAPE and c(dt=5) == DTYPE and c(dw=P + 2) == ALIGN
    for n in ("d", "rows", "pos", "w", "dr"):
        assert c(**{n: 0}) == NULL


def test_experts(lib):
    g = dict(xq=P, xs=P, T=4, tok=P, S=8, offsets=P, E=2, wq=P, ws=P, N=32, K=64, dt=0, out=P, stream=None)
    c = caller(lib.mxfp4_expert_gemm, list(g), g)
    assert c(S=-1) == SHAPE and c(T=0) == SHAPE and c(E=0) == SHAPE and c(E=513) == SHAPE and c(N=8) == SHAPE
    assert c(tok=0) == SHAPE and c(K=33) == SHAPE and c(dt=3) == DTYPE
    for n in ("xq", "xs", "offsets", "wq", "ws", "out"):
        assert c(**{n: 0}) == NULL and c(**{n: P + 2}) == ALIGN
    assert c(tok=P + 2) == ALIGN and c(S=0, T=0, xq=0, out=0) == OK
    g = dict(xq=P, xs=P, T=4, tok=P, S=8, offsets=P, E=2, wq=P, ws=P, F=32, K=64, hq=P, hs=P, stream=None)
    c = caller(lib.mxfp4_expert_swiglu, list(g), g)
    assert c(F=16) == SHAPE and c(F=0) == SHAPE and c(hq=0) == NULL and c(hs=0) == NULL and c(hs=P + 4) == ALIGN


def test_layer(lib):
    g = dict(x=P, ldx=64, dt=0, T=4, H=64, ids=P, bits=64, w=P, top=2, E=2, w13q=P, w13s=P, w2q=P, w2s=P,
             F=32, out=P, work=P, size=1 << 20, stream=None)
    c = caller(lib.mxfp4_moe, list(g), g)
    need = lib.mxfp4_moe_workspace(4, 2, 2, 64, 32, 0)
    assert need > 0 and lib.mxfp4_moe_workspace(4, 2, 2, 64, 32, 7) == 0 and lib.mxfp4_moe_workspace(0, 2, 2, 64, 32, 0) == 0
    assert c(size=need - 1) == SHAPE and c(H=48) == SHAPE and c(F=40) == SHAPE and c(E=0) == SHAPE and c(ldx=32) == SHAPE
    assert c(dt=3) == DTYPE and c(bits=8) == DTYPE
    for n in ("x", "ids", "w", "w13q", "w13s", "w2q", "w2s", "out", "work"):
        assert c(**{n: 0}) == NULL and c(**{n: P + 2}) == ALIGN
    assert c(T=0, x=0, ids=0, out=0, work=0, size=0) == OK
