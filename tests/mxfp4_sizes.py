"""Sizes that reach every kernel of the MXFP4 products on 256 compute units (test infrastructure: the GPU
tests run them, a CPU test asks the library which kernel each one takes)."""
import ctypes

CUS = 256
SWIGLU = 3

# tokens, slots per token, experts, channels: grouped rows, a third of the experts empty or nearly so
GROUPED = [(40, 2, 8, 256), (64, 4, 32, 768), (75, 2, 8, 256), (150, 4, 32, 768), (100, 2, 2, 256), (500, 2, 4, 1088),
           (500, 4, 32, 704), (1285, 2, 8, 704), (1285, 2, 8, 1344), (1285, 2, 8, 1984)]
# K with one to nine stages of 256 elements, whole and with a tail of 32 to 224; stages of 128 for K up to 1024
DEPTHS = [64, 256, 288, 512, 544, 768, 928, 1024, 1280, 1312, 2272]
# rows, channels: dense
DENSE = [(7, 144), (31, 272), (50, 1040), (150, 4112), (200, 4112), (390, 4112), (700, 4112), (1500, 4112), (4100, 4112),
         (8000, 16), (4001, 48), (1000, 64), (257, 1040)]


def form(lib, S, E, grouped, N, K, epilogue):
    """(streams, rows, channels, wavefronts) of the workgroups of a product."""
    f = lib.mxfp4_debug_form
    f.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int64]
    v = f(S, E, grouped, N, K, epilogue, CUS)
    return v >= 10 ** 9, v // 10 ** 6 % 1000, v // 1000 % 1000, v % 1000


def kernel(lib, S, E, grouped, N, K, epilogue):
    """The kernel's compiled variant but for its output type: the form and, tiled, whether K ends inside a
    stage."""
    f = form(lib, S, E, grouped, N, K, epilogue)
    stage = 128 if f == (False, 256, 128, 4) else 256
    return f + (None if f[0] else K % stage != 0,)
