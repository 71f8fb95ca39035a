"""Refusals of the block norms, the 16-bit products and the int8 product's epilogue, without a GPU: every invalid
argument gets its documented status before any HIP call (pointers here are never dereferenced)."""
import os
import re

import pytest

from quantized_gemm_quantize_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "w8a8.h")
OK, NULL, SHAPE, ALIGN, K_OVERFLOW, DTYPE, VALUE = 0, -1, -2, -3, -4, -6, -8
P = 0x10000
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("libw8a8.so not built")
    return binding.load()


def test_library_exports_every_declared_symbol(lib):
    names = set(re.findall(r"^[\w ]*\b((?:block_norm|w16a16|w8a8_gemm_act)\w*)\s*\(", open(HEADER).read(), re.M))
    assert len(names) == 10
    for fn in names:
        assert hasattr(lib, fn) and hasattr(binding, fn), fn


def test_header_constants_match_binding():
    text = open(HEADER).read()
    for name in ("W16A16_MAX_WIDTH", "BLOCK_NORM_MAX_H"):
        assert f"#define {name} {getattr(binding, name)}" in text
    for name, code in binding.ACTIVATIONS.items():
        assert re.search(rf"W8A8_ACT_{name.upper()} = {code}\b", text)
    status = {m[0]: int(m[1]) for m in re.findall(r"W8A8_(?:ERR_)?(\w+)\s*=\s*(-?\d+)", text)}
    assert (status["NULL"], status["SHAPE"], status["ALIGN"], status["K_OVERFLOW"], status["DTYPE"],
            status["VALUE"]) == (NULL, SHAPE, ALIGN, K_OVERFLOW, DTYPE, VALUE)


def caller(f, base):
    """f with named arguments over a valid call."""
    def call(**kw):
        assert set(kw) <= set(base)
        return f(*[kw.get(n, base[n]) for n in base])
    return call


def test_gemm_act(lib):
    base = dict(xq=P, xs=P, M=4, wq=P, ws=P, N=32, K=64, bias=P, act=2, residual=P, ldr=32, out=P, stream=None)
    c = caller(lib.w8a8_gemm_act, base)
    assert c(M=-1) == SHAPE and c(N=0) == SHAPE and c(N=24) == SHAPE and c(K=0) == SHAPE and c(K=24) == SHAPE
    assert c(M=2 ** 40) == SHAPE and c(N=2 ** 40) == SHAPE and c(K=2 ** 17) == K_OVERFLOW
    assert c(act=5) == DTYPE and c(act=-1) == DTYPE
    assert c(ldr=31) == SHAPE and c(ldr=2 ** 31) == SHAPE and c(ldr=36) == ALIGN
    for n in ("xq", "xs", "wq", "ws", "out"):
        assert c(**{n: 0}) == NULL
    for n in ("xq", "xs", "wq", "ws", "out", "bias", "residual"):
        assert c(**{n: P + 8}) == ALIGN
    assert c(M=0, xq=0, xs=0, wq=0, out=0) == OK


SIZES = [dict(M=-1), dict(M=2 ** 27), dict(M=2 ** 62), dict(N=0), dict(N=-8), dict(N=12), dict(K=0), dict(K=12),
         dict(N=2 ** 20 + 8), dict(K=2 ** 20 + 8), dict(N=2 ** 62), dict(M=2 ** 26, N=2 ** 10), dict(M=2 ** 26, K=2 ** 10),
         dict(N=2 ** 20, K=2 ** 20)]


def test_linear(lib):
    base = dict(x=P, ldx=2 ** 20, M=300, w=P, N=40, K=8192, dt=0, bias=P, act=1, residual=P, ldr=2 ** 20, pre=P, out=P,
                work=P, size=1 << 40, stream=None)
    c = caller(lib.w16a16_linear, base)
    for size in SIZES:
        assert c(**size) == SHAPE, size
        assert lib.w16a16_linear_workspace(*[size.get(n, base[n]) for n in "MNK"]) == 0
    need = lib.w16a16_linear_workspace(300, 40, 8192)
    assert need > 0 and c(size=need - 1) == SHAPE and c(size=-1) == SHAPE
    assert c(dt=2) == DTYPE and c(dt=-1) == DTYPE and c(act=5) == DTYPE and c(act=-1) == DTYPE
    assert c(ldx=1016) == SHAPE and c(ldx=2 ** 31) == SHAPE and c(ldx=8196) == ALIGN
    assert c(ldr=32) == SHAPE and c(ldr=2 ** 31) == SHAPE and c(ldr=44) == ALIGN
    for n in ("x", "w", "out", "work"):
        assert c(**{n: 0}) == NULL
    for n in ("x", "w", "out", "work", "bias", "residual", "pre"):
        assert c(**{n: P + 8}) == ALIGN
    # one row has no workspace, and asks for none
    assert lib.w16a16_linear_workspace(1, 40, 8192) == 0 and c(M=1, work=0, size=0, out=0) == NULL
    assert lib.w16a16_linear_workspace(0, 40, 8192) == 0
    assert c(M=0, x=0, w=0, out=0, residual=0, bias=0, pre=0, work=0, size=0) == OK


def test_linear_backward(lib):
    base = dict(d=P, ldd=2 ** 20, x=P, ldx=2 ** 20, w=P, pre=P, M=5000, N=40, K=1024, dt=1, act=2, d_pre=P, d_x=P, d_w=P,
                d_bias=P, work=P, size=1 << 40, stream=None)
    c = caller(lib.w16a16_linear_backward, base)
    for size in SIZES:
        assert c(**size) == SHAPE, size
        assert lib.w16a16_linear_backward_workspace(*[size.get(n, base[n]) for n in "MNK"]) == 0
    need = lib.w16a16_linear_backward_workspace(5000, 40, 1024)   # (300 rows need none)
    assert lib.w16a16_linear_backward_workspace(300, 40, 1024) == 0
    assert need > 0 and c(size=need - 1) == SHAPE
    assert c(dt=2) == DTYPE and c(act=5) == DTYPE and c(act=-3) == DTYPE
    assert c(ldd=32) == SHAPE and c(ldx=1016) == SHAPE and c(ldd=2 ** 31) == SHAPE and c(ldx=2 ** 31) == SHAPE
    assert c(ldd=44) == ALIGN and c(ldx=1028) == ALIGN
    for n in ("d", "x", "w", "pre", "d_pre", "work"):
        assert c(**{n: 0}) == NULL, n
    for n in ("d", "x", "w", "pre", "d_pre", "d_x", "d_w", "d_bias", "work"):
        assert c(**{n: P + 8}) == ALIGN, n
    # what only an unwanted gradient reads may be absent, and what only an activation needs; the call still ends
    # here, by a pointer that is needed
    assert c(act=0, pre=0, d_pre=0, d=0) == NULL and c(d_x=0, w=0, d=0) == NULL and c(d_w=0, x=0, d=0) == NULL


NORM = dict(r=P, ldr=64, y=P, ldy=64, post=1, pw=P, gate=P, ldg=64, scale=1.0, weight=P, eps=1e-6, T=4, H=64, dt=0,
            new=P)
NORM_SIZES = [dict(T=-1), dict(T=2 ** 24), dict(T=2 ** 60), dict(H=0), dict(H=-64), dict(H=16416), dict(H=2 ** 40 + 64),
              dict(T=2 ** 23, H=4096), dict(ldr=63), dict(ldy=63), dict(ldg=63), dict(ldr=2 ** 31), dict(ldy=2 ** 31),
              dict(ldg=2 ** 31)]


@pytest.mark.parametrize("name,outputs,multiple", [("block_norm", ("out",), 1), ("block_norm_w8a8", ("xq", "xs"), 16),
                                                   ("block_norm_mxfp4", ("codes", "scales"), 32)])
def test_norms(lib, name, outputs, multiple):
    c = caller(getattr(lib, name), {**NORM, **{n: P for n in outputs}, "stream": None})
    for size in NORM_SIZES:
        assert c(**{"ldr": 2 ** 20, "ldy": 2 ** 20, "ldg": 2 ** 20, **size}) == SHAPE, size
    assert c(dt=3) == DTYPE and c(dt=-1) == DTYPE
    for v in (INF, -INF, NAN):
        assert c(scale=v) == VALUE and c(eps=v) == VALUE
    assert c(eps=0.0) == VALUE and c(eps=-1e-6) == VALUE
    if multiple > 1:
        assert c(H=64 - multiple // 2) == SHAPE
    for n in ("r", "new", *outputs):
        assert c(**{n: 0}) == NULL, n
    for n in ("r", "y", "new", "gate"):
        assert c(**{n: P + 1}) == ALIGN and c(dt=2, **{n: P + 2}) == ALIGN, n
    for n in ("weight", "pw", *(outputs if multiple > 1 else ())):
        assert c(**{n: P + 8}) == ALIGN, n
    assert c(ldg=0, gate=P + 8) == ALIGN      # a vector
    assert c(T=0, r=0, new=0, **{n: 0 for n in outputs}) == OK
    # without a block output, what belongs to it is not looked at; the call ends by the missing output
    assert c(y=0, new=0, gate=P + 1, ldg=1, **{outputs[-1]: 0}) == NULL


def test_norm_backward(lib):
    base = dict(d_out=P, ldo=64, d_new=P, ldn=64, r=P, ldr=64, y=P, ldy=64, post=1, pw=P, gate=P, ldg=64, scale=1.0, weight=P,
                eps=1e-6, T=4, H=64, dt=0, d_r=P, d_y=P, d_gate=P, d_w=P, d_pw=P, work=P, size=1 << 40, stream=None)
    c = caller(lib.block_norm_backward, base)
    for size in [*NORM_SIZES, dict(ldo=63), dict(ldn=63), dict(ldo=2 ** 31), dict(ldn=2 ** 31)]:
        strides = dict.fromkeys(("ldo", "ldn", "ldr", "ldy", "ldg"), 2 ** 20)
        assert c(**{**strides, **size}) == SHAPE, size
    need = lib.block_norm_backward_workspace(4, 64)
    assert need >= 4 * 3 * 64 and c(size=need - 1) == SHAPE
    assert lib.block_norm_backward_workspace(0, 64) == 0 and lib.block_norm_backward_workspace(-1, 64) == 0
    assert lib.block_norm_backward_workspace(4, 16400) == 0
    assert c(dt=3) == DTYPE
    for v in (INF, NAN):
        assert c(scale=v) == VALUE and c(eps=v) == VALUE
    assert c(eps=0.0) == VALUE
    for n in ("d_out", "r", "d_r", "d_y", "work"):
        assert c(**{n: 0}) == NULL, n
    for n in ("d_out", "d_new", "r", "y", "gate", "d_r", "d_y", "d_gate"):
        assert c(**{n: P + 1}) == ALIGN and c(dt=2, **{n: P + 2}) == ALIGN, n
    for n in ("weight", "pw", "d_w", "d_pw", "work"):
        assert c(**{n: P + 8}) == ALIGN, n
    assert c(ldg=0, gate=P + 8) == ALIGN and c(ldg=0, d_gate=P + 8) == ALIGN
    assert c(T=0, d_out=0, d_new=0, r=0, y=0, d_r=0, d_y=0, d_gate=0, d_w=0, d_pw=0, work=0, size=0) == OK


def test_workspaces_are_small(lib):
    """Partial sums of the resident workgroups only, whatever the number of rows."""
    for H in (1, 64, 1280, 4096, 16384):
        sizes = [lib.block_norm_backward_workspace(T, H) for T in (1, 100, 10 ** 4, 10 ** 6)]
        assert sizes == sorted(sizes) and sizes[0] == 12 * H and sizes[3] <= 12 * H * 768
