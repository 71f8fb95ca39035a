"""Sizes that reach every tile of the 16-bit products on 256 compute units (test infrastructure: the GPU tests run
them, a CPU test asks the library which kernel each one takes)."""
import ctypes

# rows, channels, inner: tiles of 64 x 64, 128 x 128 (one and two workgroups per CU), 256 x 128 and 256 x 256; whole
# tiles, tiles shared along the inner axis, and both in one product; whole stages of 64 and an inner axis that
# ends inside one
TILED = [(72, 8, 192), (72, 8, 136), (72, 8, 1024), (72, 8, 968), (1680, 1800, 256), (1608, 1944, 200), (1104, 760, 5824),
         (1280, 720, 5640), (3272, 1168, 3648), (1056, 3712, 3592), (1944, 1552, 192), (2192, 1352, 136),
         (1288, 1008, 8960), (1096, 1184, 8456), (3456, 2336, 640), (3384, 2392, 720), (3064, 2480, 1792),
         (3736, 1984, 1760), (1496, 1408, 8640), (968, 1504, 9872), (2960, 2696, 3328), (1184, 6736, 3088),
         (2240, 3592, 384), (2456, 3216, 344), (1984, 2560, 9664), (1504, 3536, 9544), (3048, 5512, 1792), (9408, 1760, 1776)]
# few rows: 1 to 4 groups of 16
ROWS = [(1, 8, 8), (16, 4096, 1024), (17, 1024, 4096), (32, 2048, 1024), (48, 2048, 512), (64, 4096, 520)]
FORMS = 5


def form(lib, M, N, K, forward=True):
    """("rows",) or (form, whole tiles, shared tiles, the inner axis ends inside a stage)."""
    f = lib.w16a16_debug_form
    f.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int]
    v = f(M, N, K, forward)
    if v >= 10 ** 6:
        return ("rows",)
    return v // 10 ** 5, v // 10 ** 4 % 10 == 1, v % 10 ** 4 > 1, K % 64 != 0
