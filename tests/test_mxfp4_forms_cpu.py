"""The sizes of the GPU tests reach every compiled variant of the MXFP4 products, without a GPU."""
import os
import re

import pytest

from mxfp4_sizes import DENSE, DEPTHS, GROUPED, SWIGLU, kernel
from quantized_gemm_quantize_amd import binding, build

CSRC = build.CSRC


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("libw8a8.so not built")
    return binding.load()


def launches(name, pattern):
    """Numbers of every launch of `pattern` in a kernel's file."""
    text = open(os.path.join(CSRC, name)).read()
    return {tuple(int(v) for v in m) for m in re.findall(pattern, text)}


def test_every_variant_is_reached(lib):
    tiled = {(bm, bn, gm * gn) for bm, bn, gm, gn in
             launches("mxfp4_tiled.hip", r"return launch_(?:plain|shape)<(\d+), (\d+), (\d+), (\d+), \d, \d, \d>\(op")}
    assert len(tiled) == 6
    tails = {(False, *t, tail) for t in tiled for tail in (False, True)}
    with_swiglu = {t for t in tails if t[2] > 64}             # 64 x 64 has plain outputs only
    plain, swiglu = set(), set()
    for T, top, E, N in GROUPED:
        for K in DEPTHS:
            plain.add(kernel(lib, T * top, E, 1, N, K, 2))
            swiglu.add(kernel(lib, T * top, E, 1, N, K, SWIGLU))
    # streamed: (row tiles, channels, wavefronts) as launch_rows has them
    text = open(os.path.join(CSRC, "mxfp4_decode.hip")).read()
    rows = text[text.index("hipError_t launch_rows("):text.index("hipError_t launch_fused(")]
    forms = set(re.findall(r"launch_plain<MT, (\d), (\d)>", rows))
    assert forms == {("4", "2"), ("2", "4"), ("1", "8"), ("1", "4")}  # the last two are dense
    streamed = {(True, r, 16 * int(c), int(w), None) for r in (16, 32) for c, w in forms if c != "1"}
    assert plain == tails | streamed
    assert swiglu == with_swiglu | {(True, r, 64, w, None) for r in (16, 32) for w in (2, 4)}
    dense = {kernel(lib, M, 1, 0, N, K, 2) for M, N in DENSE for K in DEPTHS}
    assert dense == tails | {(True, 16, 16, 8, None), (True, 32, 16, 8, None), (True, 64, 16, 4, None)}


@pytest.mark.parametrize("M,N,K,streams", [(8000, 16, 8192, True), (8000, 64, 1024, False), (8000, 48, 8192, False),
                                           (3000, 96, 2048, False), (1000, 256, 8192, True), (257, 1040, 1312, True),
                                           (257, 1040, 4096, False), (1000, 304, 1024, True), (1500, 304, 1024, False)])
def test_tall_narrow_layers(lib, M, N, K, streams):
    """The streaming kernel takes dense rows past 64 only while its workgroups run at once, or K is
    short (measured at these sizes, the other kernel takes up to 2.1 times as long)."""
    assert kernel(lib, M, 1, 0, N, K, 2)[0] == streams
