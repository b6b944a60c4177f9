"""More of what the cache's calls refuse, without a GPU.  Each call here has a later argument that is refused as well, so
nothing is ever launched."""
import ctypes
import math

import pytest

from weight_only_quantization_pack_amd import binding as B

NULL, SHAPE, UNSUP, ALIGN, WS = 1, 2, 3, 4, 5
P = ctypes.c_void_p(0x10000)
OUT = ctypes.c_void_p(0x20000)
NUL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    return B.load_library()


def test_scales_of_scores(lib):
    """|scale| times 2^24 has to stay in fp32: the unit of the products' operands."""
    def call(scale):
        return lib.awq_cache_attention(P, 512, P, P, P, P, P, P, P, OUT, NUL, scale, 0, 0.0, 8, 4, 2, 4, 2, 128, 9, 16, 4,
                                       20000, 0, P, 0, NUL)
    for good in (0.0, -1.0, 2.0 ** -130, 2.0 ** 99, -2.0 ** 99):
        assert call(good) == WS, good
    for bad in (2.0 ** 100, -2.0 ** 100, 2.0 ** 105, 3e38, math.inf, math.nan):
        assert call(bad) == UNSUP, bad
