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


def test_alignment_of_copied_pages(lib):
    """Pages that are no multiple of 16 bytes (scales of 1, 2, 3, 5 .. heads, and any layer's slice of them) are copied in
    words of 4; others need 16."""
    def call(address, size, pairs=NUL):
        return lib.awq_cache_copy_pages((ctypes.c_void_p * 1)(address), (ctypes.c_size_t * 1)(size), 1, 1, pairs, NUL, 4, 9, NUL)
    for size in (4, 12, 20, 24, 8200):
        for address in (0x10000, 0x10004, 0x10008, 0x1000C):
            assert call(address, size) == NULL, (address, size)          # as far as the pairs, which are missing
        for address in (0x10001, 0x10002, 0x10006):
            assert call(address, size) == ALIGN, (address, size)
    for size in (16, 32, 8192):
        assert call(0x10010, size) == NULL
        for address in (0x10004, 0x10008):
            assert call(address, size) == ALIGN, (address, size)
