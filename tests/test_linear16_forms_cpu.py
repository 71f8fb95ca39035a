"""The sizes of the GPU tests reach every compiled variant of the 16-bit products, without a GPU."""
import os
import re

import pytest

from linear16_sizes import D_W, D_X, FORMS, PAIR_D_W, PAIR_D_X, PAIRS, ROWS, TILED, form
from quantized_gemm_quantize_amd import binding, build


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("libw8a8.so not built")
    return binding.load()


def test_every_tile_is_reached(lib):
    text = open(os.path.join(build.CSRC, "linear16_tiled.hip")).read()
    one = text[text.index("hipError_t launch_form("):text.index("hipError_t launch_pair_form(")]
    assert len(re.findall(r"return launch<F16, |return launch_deep<F16, ", one)) == FORMS
    # as the forward product, as d_x of a layer of that inner axis, as d_w of one of as many rows
    for reached in ({form(lib, *size) for size in TILED}, {form(lib, m, k, n, D_X) for m, n, k in TILED},
                    {form(lib, k, m, n, D_W) for m, n, k in TILED}):
        assert {r[0] for r in reached} == set(range(FORMS))
        for f in range(FORMS):
            for tail in (False, True):
                # all tiles whole, all shared, and some of each where a round of tiles does not hold them all
                assert (f, True, False, tail) in reached and (f, False, True, tail) in reached
                assert f == 0 or (f, True, True, tail) in reached


def test_every_tile_of_both_gradients_is_reached(lib):
    text = open(os.path.join(build.CSRC, "linear16_tiled.hip")).read()
    both = text[text.index("hipError_t launch_pair_form("):text.index("hipError_t launch_type(")]
    assert len(re.findall(r"return launch_both<F16, ", both)) == 3
    reached = {(form(lib, *size, PAIR_D_X), form(lib, *size, PAIR_D_W), size[0] >= size[1]) for size in PAIRS}
    assert all(x[0] == w[0] for x, w, _ in reached)
    for f in (0, 2, 4):
        for first in (False, True):      # d_w first, of more rows than channels
            for tx in (False, True):
                for tw in (False, True):
                    of = {(x[1:3], w[1:3]) for x, w, order in reached if (x[0], x[3], w[3], order) == (f, tx, tw, first)}
                    assert ((True, False), (True, False)) in of, (f, first, tx, tw)
            of = {(x[1:3], w[1:3]) for x, w, order in reached if (x[0], order) == (f, first)}
            assert any((w if first else x) == (False, True) for x, w in of)      # the first one's tiles shared
            assert f == 0 or any((x if first else w) == (True, True) for x, w in of)   # the second one's last


def test_few_rows(lib):
    assert {-(-m // 16) for m, _, _ in ROWS} == {1, 2, 3, 4}
    assert all(form(lib, *size) == ("rows",) for size in ROWS)
    # past 16 rows only where few workgroups of it run one after the other
    assert form(lib, 16, 65536, 4096) == ("rows",) and form(lib, 17, 65536, 4096) != ("rows",)
    assert form(lib, 65, 64, 64) != ("rows",)


def test_workspaces_hold_the_shared_tiles(lib):
    tile = [64 * 64, 128 * 128, 128 * 128, 256 * 128, 256 * 256, 64 * 64]
    sides = [(64, 64), (128, 128), (128, 128), (256, 128), (256, 256), (64, 64)]
    for m, n, k in TILED:
        f, whole, shared, _ = form(lib, m, n, k)
        need = lib.w16a16_linear_workspace(m, n, k)
        if not shared:
            assert need == 0
            continue
        bm, bn = sides[f]
        tiles = -(-m // bm) * -(-n // bn)
        slots = [768, 256, 512, 256, 256, 256][f]
        rest = tiles % slots if whole else tiles
        assert need % (4 * tile[f] * rest) == 0 and 2 <= need // (4 * tile[f] * rest) <= 64
        assert lib.w16a16_linear_workspace(m, n, k + 4) == 0      # a refused size


def test_plans_of_the_largest_and_smallest_sizes(lib):
    """Every plan has whole numbers of tiles and a workspace that fits the sums it needs, up to the limits."""
    sizes = [(1, 8, 8), (16, 2 ** 20, 2 ** 15), (17, 8, 8), (2 ** 27 - 1, 8, 8), (2 ** 27 - 1, 256, 256), (2 ** 15, 2 ** 20, 8),
             (2 ** 15, 8, 2 ** 20), (2 ** 15, 2 ** 20, 2 ** 15), (17, 2 ** 20, 2 ** 15), (64, 2 ** 15, 2 ** 20), (2 ** 20, 2 ** 15, 2 ** 15)]
    for m, n, k in sizes:
        forward = lib.w16a16_linear_workspace(m, n, k)
        assert 0 <= forward <= 2 ** 31 and (m > 16 or forward == 0)
        assert 0 <= lib.w16a16_linear_backward_workspace(m, n, k) <= 2 ** 31
        assert form(lib, m, n, k) is not None
        for product in (D_X, D_W, PAIR_D_X, PAIR_D_W):
            f, whole, shared, _ = form(lib, m, n, k, product)
            assert 0 <= f < FORMS and (whole or shared), (m, n, k, product)
        assert form(lib, m, n, k, PAIR_D_X)[0] == form(lib, m, n, k, PAIR_D_W)[0]
