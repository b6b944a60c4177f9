"""Infinities and NaN among what goes into the cache and out of it: a block's scale carries them, and only
the queries that see one of the block's tokens."""
import numpy as np
import pytest

import weight_only_quantization_pack_amd as awq

import block_reference as R
import cache_reference as C
from cache_util import Case, gpu as put, host_cache
from gpu_util import announce

pytestmark = pytest.mark.gpu

BAD = [float("nan"), float("inf"), -float("inf")]


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("bad", BAD, ids=str)
def test_append(gpu, page, bad):
    """A block with such a token has a scale that is not finite and reads as NaN; every other block is as without it."""
    announce("append", bad, page)
    case = Case([(40, 3), (20, 11), (1, page - 1)], 4, 2, 64, page, "bf16", seed=page)
    k, v = case.rows(2), case.rows(2)
    caches = []
    for hurt in (False, True):
        cache, tables, lens, st = case.on_gpu()
        if hurt:
            k[7, 1, 5] = bad                     # sequence 0, position 10, head 1
            v[45, 0, 63] = bad                   # sequence 1, position 16, head 0
        awq.cache_append(None, k, v, cache, tables, lens, st)
        caches.append(host_cache(cache))
        got = awq.cache_read(cache, tables, lens, st, tokens=case.T, dtype=case.dtype)
    where = {0: (int(case.tables[0, 10 // page]), 1), 1: (int(case.tables[1, 16 // page]), 0)}
    for i in range(2):
        codes, scales = caches[1][2 * i:2 * i + 2]
        assert not np.isfinite(scales[where[i]])
        others = np.ones(scales.shape, bool)
        others[where[i]] = False
        assert np.array_equal(scales[others], caches[0][2 * i + 1][others])
        assert np.array_equal(codes[others], caches[0][2 * i][others])
        for t, (b, pos) in enumerate(C.places(case.starts, case.lens, case.T)):
            for h in range(2):
                inside = (int(case.tables[b, pos // page]), h) == where[i]
                assert bool(got[i][t, h].isnan().all()) == inside and bool(got[i][t, h].isfinite().all()) != inside
    # the next token of the block finds it so; one that starts the page anew does not
    cache = tuple(put(c) for c in caches[1])
    p, h = where[0]
    tables = np.full((2, 1), p, np.int32)
    awq.cache_append(None, k[:1], v[:1], cache, put(tables[:1]), put(np.array([12], np.int32)))
    assert not np.isfinite(host_cache(cache)[1][p, h])
    awq.cache_append(None, k[:1], v[:1], cache, put(tables[:1]), put(np.array([1], np.int32)))
    assert np.isfinite(host_cache(cache)[1][p]).all()


def attend(case, cache, q, st, **kw):
    import torch
    lse = torch.empty(case.T, case.heads, device="cuda")
    out = awq.cache_attention(q, tuple(put(c) for c in cache), put(case.tables), put(case.lens), st, lse=lse, **kw)
    return R.to_f64(out), lse.cpu().numpy()


@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("pairs,page,dim,max_len", [([(1, 100), (1, 40), (1, 200)], 16, 128, None),
                                                    ([(1, 4000), (1, 300)], 64, 64, None), ([(1, 250)], 32, 96, 256),
                                                    ([(7, 900), (3, 20)], 16, 256, None),
                                                    ([(150, 60), (300, 0), (90, 2000)], 64, 128, None),
                                                    ([(120, 500)], 16, 192, None)], ids=str)
@pytest.mark.parametrize("bad", BAD[:2], ids=str)
def test_attention(gpu, pairs, page, dim, max_len, window, bad):
    """Blocks of keys and of values; queries that see a token of theirs have NaN, all others the same bits as before."""
    announce("attention", pairs, page, dim, window, bad)
    case = Case(pairs, 4, 2, dim, page, seed=page + dim)
    q = case.rows(4)
    st = put(case.starts) if case.T != len(pairs) else None
    kw = dict(window=window, softcap=30.0 if page == 32 else 0.0, max_len=max_len)
    clean, clean_lse = attend(case, case.cache, q, st, **kw)
    assert np.isfinite(clean).all() and np.isfinite(clean_lse).all()
    for tensor in (1, 3):
        for last in (False, True):               # a block in the middle, and the one that is being filled
            cache = [c.copy() for c in case.cache]
            hurt = []
            for b, n in enumerate(case.lens):
                w = (int(n) - 1) // page if last else int(n) // (2 * page)
                cache[tensor][case.tables[b, w], b % 2] = bad
                hurt.append((w * page, min((w + 1) * page, int(n)) - 1))
            out, lse = attend(case, cache, q, st, **kw)
            for t, (b, pos) in enumerate(C.places(case.starts, case.lens, case.T)):
                first, end = hurt[b]
                sees = first <= pos and (not window or pos - window < end)
                for h in range(4):
                    if sees and h // 2 == b % 2:
                        assert np.isnan(out[t, h]).all() and np.isnan(lse[t, h]), (t, h)
                    else:
                        assert np.array_equal(out[t, h], clean[t, h]) and lse[t, h] == clean_lse[t, h], (t, h)


@pytest.mark.parametrize("pairs", [[(1, 90), (1, 3000)], [(130, 200)]], ids=str)
def test_queries(gpu, pairs):
    """A query that is not finite makes its own row and head NaN.  The others' bits may change with it: rows of a
    tile raise their running maximum together, and the weights are rounded relative to it.  Their bound holds for
    every such choice (it counts a maximum up to 2^2 below the largest weight)."""
    announce("attention queries", pairs)
    case = Case(pairs, 4, 2, 128, 32, seed=3)
    q = case.rows(4)
    ref, ref_lse, bound = C.attention(R.to_f64(q), case.cache, case.tables, case.lens, case.starts, 128 ** -0.5)
    bound = bound + R.unit(q.dtype) * (np.abs(ref) + bound) + 2.0 ** -24
    q[0, 1, 77], q[-1, 2, 0] = float("nan"), float("inf")
    out, lse = attend(case, case.cache, q, put(case.starts))
    for t in range(case.T):
        for h in range(4):
            if (t, h) in ((0, 1), (case.T - 1, 2)):
                assert np.isnan(out[t, h]).all()
            else:
                assert np.all(np.abs(out[t, h] - ref[t, h]) <= bound[t, h])
                assert abs(lse[t, h] - ref_lse[t, h]) <= 1e-3 + 2.0 ** -20 * abs(ref_lse[t, h])
