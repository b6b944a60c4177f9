"""Rotary positions and the paged cache without a GPU: what the calls refuse, before
anything is launched, and the frequencies, which are computed on the host."""
import ctypes
import math

import numpy as np
import pytest

import weight_only_quantization_pack_amd as awq
from weight_only_quantization_pack_amd import binding as B

import cache_reference as C

OK, NULL, SHAPE, UNSUP, ALIGN, WS = 0, 1, 2, 3, 4, 5
P, P2, P3, P4, P5 = (ctypes.c_void_p(0x10000 * i) for i in range(1, 6))     # never used
MIS, ODD, NUL = ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10002), ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    return B.load_library()


@pytest.mark.parametrize("rotary", [2, 16, 64, 128, 512])
@pytest.mark.parametrize("scaling", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=2.5),
                                     dict(scaling="yarn", factor=16.0, original_length=4096.0, low=1.0, high=32.0),
                                     dict(scaling="bands", factor=8.0, original_length=8192.0, low=1.0, high=4.0)])
def test_frequencies(rotary, scaling):
    if scaling.get("scaling") == "base" and rotary == 2:
        with pytest.raises(B.AwqError):
            awq.rope_frequencies(rotary, 10000.0, device="cpu", **scaling)
        return
    got, magnitude = awq.rope_frequencies(rotary, 500000.0, device="cpu", **scaling)
    k = dict(scaling)
    want, m = C.frequencies(rotary, 500000.0, k.pop("scaling", None), k.pop("factor", 1.0), k.pop("original_length", 0.0), **k)
    # fp32 of a 64-bit value: half a step, and the few of 64 bits that logarithms cost
    assert np.all(np.abs(got.double().numpy() - want) <= (2.0 ** -24 + 1e-12) * want)
    assert abs(magnitude - m) <= 2.0 ** -24 * m


def test_frequencies_refused(lib):
    out, m = (ctypes.c_float * 256)(), ctypes.c_float()

    def call(rotary=64, base=1e4, scaling=0, factor=1.0, original=4096.0, low=1.0, high=32.0, f=out, mag=ctypes.byref(m)):
        return lib.awq_rope_frequencies(rotary, base, scaling, factor, original, low, high, f, mag)
    assert call() == OK and call(scaling=3, factor=2.0) == OK
    assert call(f=NUL) == NULL and call(mag=NUL) == NULL
    for bad in (dict(rotary=0), dict(rotary=63), dict(rotary=514), dict(rotary=2, scaling=2, factor=2.0)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(base=1.0), dict(base=math.nan), dict(base=math.inf), dict(scaling=5), dict(scaling=-1),
                dict(scaling=1, factor=0.5), dict(scaling=1, factor=math.inf), dict(scaling=3, factor=2.0, original=0.0),
                dict(scaling=4, factor=2.0, low=2.0, high=2.0), dict(scaling=4, factor=2.0, low=0.0)):
        assert call(**bad) == UNSUP, bad
    with pytest.raises(ValueError):
        awq.rope_frequencies(64, scaling="other", device="cpu")


def test_rope_validation(lib):
    def call(x=P, xs=512, pos=P2, f=P3, m=1.0, out=P4, os=512, T=4, heads=4, dim=128, rotary=128, layout=0, inverse=0,
             dtype=0):
        return lib.awq_rope(x, xs, pos, f, m, out, os, T, heads, dim, rotary, layout, inverse, dtype, NUL)
    for name in ("x", "pos", "f", "out"):
        assert call(**{name: NUL}) == NULL, name
    for bad in (dict(x=MIS), dict(out=MIS), dict(pos=ODD), dict(f=ODD)):
        assert call(**bad) == ALIGN, bad
    for bad in (dict(T=-1), dict(heads=0), dict(dim=0), dict(dim=120), dict(dim=528), dict(rotary=0), dict(rotary=24),
                dict(rotary=144), dict(xs=504), dict(xs=516), dict(os=500), dict(T=(1 << 31) - 1),
                dict(heads=65536, xs=1 << 24, os=1 << 24)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(layout=2), dict(inverse=2), dict(dtype=2), dict(m=math.nan)):
        assert call(**bad) == UNSUP, bad
    assert call(T=0, x=NUL, f=NUL) == OK


def cache_calls(lib):
    """append, read and attention with the same cache and sequences"""
    def append(q=P, qs=512, k=P2, ks=256, v=P3, vs=256, out=P4, f=P5, m=1.0, rotary=64, layout=0, kc=P, ksc=P2, vc=P3,
               vsc=P4, tables=P, lens=P2, starts=P3, T=8, B=4, W=2, heads=4, kv=2, dim=128, pages=9, page=16, dtype=0):
        return lib.awq_cache_append(q, qs, k, ks, v, vs, out, f, m, rotary, layout, kc, ksc, vc, vsc, tables, lens, starts,
                                    T, B, W, heads, kv, dim, pages, page, dtype, NUL)

    def read(kc=P, ksc=P2, vc=P3, vsc=P4, tables=P, lens=P2, starts=P3, T=8, B=4, W=2, kv=2, dim=128, pages=9, page=16,
             dtype=0, k=P4, v=P5):
        return lib.awq_cache_read(kc, ksc, vc, vsc, tables, lens, starts, T, B, W, kv, dim, pages, page, dtype, k, v, NUL)

    def attention(q=P, qs=512, kc=P, ksc=P2, vc=P3, vsc=P4, tables=P, lens=P2, starts=P3, out=P5, lse=NUL, scale=0.1,
                  window=0, cap=0.0, T=8, B=4, W=2, heads=4, kv=2, dim=128, pages=9, page=16, new=4, most=20000, dtype=0,
                  ws=P, ws_bytes=1 << 40):
        return lib.awq_cache_attention(q, qs, kc, ksc, vc, vsc, tables, lens, starts, out, lse, scale, window, cap, T, B, W,
                                       heads, kv, dim, pages, page, new, most, dtype, ws, ws_bytes, NUL)
    return append, read, attention


def test_cache_calls_validation(lib):
    append, read, attention = cache_calls(lib)
    for call in (append, read, attention):
        for name in ("kc", "ksc", "vc", "vsc", "tables", "lens"):
            assert call(**{name: NUL}) == NULL, name
        for bad in (dict(kc=MIS), dict(vc=MIS), dict(ksc=ODD), dict(vsc=ODD), dict(tables=ODD), dict(lens=ODD), dict(starts=ODD)):
            assert call(**bad) == ALIGN, bad
        for bad in (dict(T=-1), dict(B=-1), dict(W=0), dict(kv=0), dict(pages=0), dict(pages=(1 << 30) + 1),
                    dict(T=(1 << 20) + 1), dict(B=(1 << 20) + 1), dict(starts=NUL, T=5)):
            assert call(**bad) == SHAPE, bad
        for bad in (dict(page=8), dict(page=48), dict(page=256), dict(dim=80), dict(dim=32), dict(dim=512), dict(dtype=2)):
            assert call(**bad) == UNSUP, bad
        assert call(T=0) == OK and call(B=0) == OK and call(T=0, B=0, starts=NUL) == OK
    for bad in (dict(k=NUL), dict(v=NUL), dict(out=NUL)):
        assert append(**bad) == NULL, bad
    for bad in (dict(q=MIS), dict(k=MIS), dict(v=MIS), dict(out=MIS), dict(f=ODD)):
        assert append(**bad) == ALIGN, bad
    for bad in (dict(qs=504), dict(ks=248), dict(vs=260), dict(rotary=0), dict(rotary=136), dict(rotary=144), dict(heads=0),
                dict(T=1 << 20, kv=256, ks=1 << 15, vs=1 << 15), dict(heads=65536, qs=1 << 24)):
        assert append(**bad) == SHAPE, bad
    for bad in (dict(layout=2), dict(m=math.inf)):
        assert append(**bad) == UNSUP, bad
    assert append(f=NUL, rotary=-1, layout=9, T=0) == OK              # no rotation: its arguments are not looked at
    assert read(k=NUL) == NULL and read(v=MIS) == ALIGN
    assert attention(q=NUL) == NULL and attention(out=MIS) == ALIGN and attention(lse=ODD) == ALIGN
    for bad in (dict(heads=0), dict(heads=5), dict(new=0), dict(most=0), dict(qs=504), dict(T=1 << 20, heads=16, qs=1 << 15)):
        assert attention(**bad) == SHAPE, bad
    for bad in (dict(scale=math.nan), dict(window=-1), dict(cap=-1.0), dict(cap=math.inf)):
        assert attention(**bad) == UNSUP, bad
    need = lib.awq_cache_attention_workspace_bytes(8, 4, 4, 2, 128, 4, 20000)
    assert need > 0 and attention(ws=NUL) == NULL and attention(ws=MIS) == ALIGN and attention(ws_bytes=need - 1) == WS
    size = lib.awq_cache_attention_workspace_bytes
    assert size(8, 4, 4, 2, 128, 4, 64) == size(0, 4, 4, 2, 128, 4, 20000) == size(8, 4, 5, 2, 128, 4, 20000) == 0


def test_book_validation(lib):
    def fork(t=P, l=P2, r=P3, p=P4, ot=P5, ol=P, B=4, n=4, W=2, pages=9, page=16):
        return lib.awq_cache_fork(t, l, r, p, ot, ol, B, n, W, pages, page, NUL)

    def reserve(t=P, l=P2, r=P3, c=P4, pr=P5, s=P, B=4, W=2, pages=9, page=16):
        return lib.awq_cache_reserve(t, l, r, c, pr, s, B, W, pages, page, NUL)

    def compact(t=P, l=P2, r=P3, m=P4, c=P5, B=4, W=2, pages=9, page=16):
        return lib.awq_cache_compact(t, l, r, m, c, B, W, pages, page, NUL)
    for call, names in ((fork, ("t", "l", "r", "p", "ot", "ol")), (reserve, ("t", "l", "r", "c", "pr", "s")),
                        (compact, ("t", "l", "r", "m", "c"))):
        for name in names:
            assert call(**{name: NUL}) == NULL, name
            assert call(**{name: ODD}) == ALIGN, name
        for bad in (dict(B=-1), dict(B=65536), dict(W=0), dict(pages=0), dict(pages=(1 << 30) + 1),
                    dict(B=4096, W=1 << 19)):
            assert call(**bad) == SHAPE, bad
        assert call(page=24) == UNSUP
    assert fork(n=-1) == SHAPE and fork(ot=P) == UNSUP and fork(B=0, n=0, r=NUL) == OK
    assert reserve(B=4097) == UNSUP

    def copy(tensors=(0x10000, 0x20000), sizes=(64, 8), n=None, layers=1, pairs=P, count=NUL, most=4, pages=9):
        k = max(len(tensors), 1)
        return lib.awq_cache_copy_pages((ctypes.c_void_p * k)(*tensors), (ctypes.c_size_t * k)(*sizes),
                                        len(tensors) if n is None else n, layers, pairs, count, most, pages, NUL)
    assert copy(tensors=(0x10000, None)) == NULL and copy(pairs=NUL) == NULL
    assert copy(tensors=(0x10008, 0x20000)) == ALIGN and copy(pairs=ODD) == ALIGN and copy(count=ODD) == ALIGN
    for bad in (dict(sizes=(64, 6)), dict(sizes=(0, 4)), dict(layers=0), dict(most=-1), dict(pages=0)):
        assert copy(**bad) == SHAPE, bad
    assert copy(n=0) == UNSUP and copy(tensors=(0x10000,) * 9, sizes=(16,) * 9) == UNSUP
    assert copy(most=0, pairs=NUL) == OK
    assert lib.awq_cache_copy_pages(NUL, NUL, 1, 1, P, NUL, 4, 9, NUL) == NULL


def test_binding_refuses_tensors_off_the_gpu():
    import torch
    x = torch.zeros(2, 4, 64, dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(2, 3, dtype=torch.int32)
    cache = awq.empty_cache(4, 2, 16, 64, device="cpu")
    freq, _ = awq.rope_frequencies(64, device="cpu")
    for call in (lambda: awq.rope(x, i, freq), lambda: awq.cache_append(x, x[:, :2], x[:, 2:], cache, t, i),
                 lambda: awq.cache_read(cache, t, i), lambda: awq.cache_attention(x, cache, t, i),
                 lambda: awq.cache_fork(t, i, i, i, 16), lambda: awq.cache_reserve(t, i, i, i, 16),
                 lambda: awq.cache_compact(t, i, i, 16), lambda: awq.cache_copy_pages(cache, t)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_refusals_of_what_cannot_be_right(lib):
    """Overlapping rows of different strides, outputs over inputs, caps and lengths outside what is computed rightly."""
    out, m = (ctypes.c_float * 256)(), ctypes.c_float()
    for scaling in (3, 4):
        for original, high in ((math.inf, 32.0), (4096.0, math.inf), (math.nan, 32.0), (4096.0, math.nan)):
            assert lib.awq_rope_frequencies(64, 1e4, scaling, 2.0, original, 1.0, high, out, ctypes.byref(m)) == UNSUP
    assert lib.awq_rope(P, 1024, P2, P3, 1.0, P, 512, 4, 4, 128, 128, 0, 0, 0, NUL) == UNSUP
    append, _, attention = cache_calls(lib)
    assert append(out=P, qs=1024) == UNSUP
    assert attention(out=P) == UNSUP
    for cap in (1e-30, 2.0 ** -11, 1025.0, 1e30, math.nan):
        assert attention(cap=cap) == UNSUP, cap
    assert lib.awq_cache_fork(P, P2, P3, P4, P5, P2, 4, 4, 2, 9, 16, NUL) == UNSUP
