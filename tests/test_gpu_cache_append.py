"""GPU parity of awq_cache_append and awq_cache_read against 64 bits.

Scales: max|x| / 127 of fp32 rows that a turn left within 2^-20.5 (|a| + |b|): 2^-19 relative to the block's
maximum with room.  Codes: half a step, and what the value and the scale are off by in steps (|x / s| <= 127):
127 * 2^-18.  The codes that were there: exact integers times a fp32 quotient, half a step and 127 * 2^-18 again.
"""
import numpy as np
import pytest

import weight_only_quantization_pack_amd as awq

import block_reference as R
import cache_reference as C
from cache_util import DTYPES, Case, freq, gpu as put, host_cache, ints
from gpu_util import announce, guarded_empty, sentinel_intact

pytestmark = pytest.mark.gpu

SLACK = 127 * 2.0 ** -18


def check_blocks(before, after, x, case, where):
    """The cache's codes and scales after x went in; everything else as before."""
    codes, scales = after
    want = C.append(x, before[0], before[1], case.tables, where, case.page)
    kept_codes, kept_scales = before[0].copy(), before[1].copy()
    for (p, h), (scale, slots) in want.items():
        assert abs(scales[p, h] - scale) <= 2.0 ** -19 * scale, (p, h, scales[p, h], scale)
        for s, exact in slots.items():
            assert np.abs(codes[p, h, s] - exact).max() <= 0.5 + SLACK, (p, h, s)
            kept_codes[p, h, s] = codes[p, h, s]
        kept_scales[p, h] = scales[p, h]
    assert np.array_equal(kept_codes, codes) and np.array_equal(kept_scales, scales)


def run(case, layout="half", rotary=None, base=10000.0, queries=True, starts=True, spread=1.0):
    import torch
    cache, tables, lens, st = case.on_gpu()
    qkv = case.rows(case.heads + 2 * case.kv, spread)
    h, kv = case.heads, case.kv
    q, k, v = qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:]
    f, m = (None, 1.0) if rotary == 0 else freq(rotary or case.dim, base)
    out, raw, n = guarded_empty((case.T, h, case.dim), case.dtype)
    out.fill_(-3.0)
    got = awq.cache_append(q if queries else None, k, v, cache, tables, lens, st if starts else None, inv_freq=f,
                           layout=layout, magnitude=m, out=out if queries else None)
    torch.cuda.synchronize()
    assert sentinel_intact(raw, n)
    where = C.places(case.starts, case.lens, case.T)
    pos = np.array([p for _, p in where])
    turn = (lambda x: R.to_f64(x)) if f is None else lambda x: C.rope(R.to_f64(x), pos, f.cpu().numpy(), m, layout)
    after = host_cache(cache)
    check_blocks(case.cache[:2], after[:2], turn(k), case, where)
    check_blocks(case.cache[2:], after[2:], R.to_f64(v), case, where)
    if queries:
        ref = turn(q)
        a = R.to_f64(q)
        pair = np.abs(a).max(-1, keepdims=True) * 2
        assert np.all(np.abs(R.to_f64(got) - ref) <= R.unit(got.dtype) * np.abs(ref) + 2.0 ** -20.5 * pair + 2.0 ** -24)
    else:
        assert got is None
    # and read back: code * scale rounded once
    ks, vs = awq.cache_read(cache, tables, lens, st if starts else None, tokens=case.T, dtype=case.dtype)
    for got, (codes, scales) in ((ks, after[:2]), (vs, after[2:])):
        ref = C.read(codes, scales, case.tables, where, case.page)
        assert np.all(np.abs(R.to_f64(got) - ref) <= (R.unit(got.dtype) + 2.0 ** -23) * np.abs(ref) + 2.0 ** -25)
    return cache


# one token, a full page, one more; pages that end inside; several sequences, empty ones, long pasts
SEQS = [[(1, 0)], [(1, 15)], [(1, 16)], [(17, 0)], [(3, 5), (40, 0), (1, 31), (0, 9), (2, 62)], [(0, 0), (5, 130), (0, 3)],
        [(130, 7), (1, 64)], [(300, 21)]]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("pairs", SEQS, ids=str)
def test_append(gpu, pairs, page):
    announce("append", pairs, page)
    run(Case(pairs, 4, 2, 64, page, seed=len(pairs) + page))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,kv,dim,rotary", [(1, 1, 64, 64), (8, 8, 96, 48), (10, 2, 128, 64), (6, 3, 192, 192), (4, 1, 256, 256),
                                                 (7, 1, 128, 0), (2, 2, 256, 32)])
def test_heads_and_types(gpu, heads, kv, dim, rotary, dtype, layout):
    announce("append heads", heads, kv, dim, rotary, dtype, layout)
    for page in (16, 128):
        run(Case([(5, 11), (140, 3), (1, 0)], heads, kv, dim, page, dtype, seed=dim + heads), layout, rotary, 500000.0)


def test_decode_rows(gpu):
    """One row for each sequence without starts; without queries; an empty sequence and one past its table."""
    announce("append decode")
    pairs = [(1, n) for n in (0, 1, 15, 16, 31, 77)]
    run(Case(pairs, 8, 2, 128, 16, seed=1), starts=False)
    run(Case(pairs, 8, 2, 128, 32, "bf16", seed=2), queries=False)
    lens = [1, 0, 16, 17, 32, 400]                       # sequence 1 holds nothing, sequence 5 more than its table
    run(Case(pairs, 8, 2, 128, 16, seed=3, lens=lens), starts=False)


def test_scales_grow_and_stay(gpu):
    """Tokens one by one: what a block holds follows its scale."""
    announce("append token by token")
    for spread in (0.02, 30.0):                          # under and far over the scales that are there
        case = Case([(1, 5), (1, 31)], 2, 2, 64, 32, seed=4)
        for _ in range(6):
            cache = run(case, spread=spread)
            case.cache = host_cache(cache)
            grown = [(1, int(n)) for n in case.lens]
            lens = case.lens + 1
            if -(-int(lens.max()) // case.page) > case.tables.shape[1]:
                break
            case.lens = lens


def test_zeros_bad_pages_and_rows_behind(gpu):
    import torch
    announce("append zeros, bad pages, rows behind the last sequence")
    case = Case([(20, 8), (40, 0)], 2, 2, 64, 16, seed=5, bad=[(0, 1, 1 << 30), (1, 0, -1), (1, 2, 10 ** 6)])
    run(case)
    case = Case([(4, 0), (3, 20)], 2, 2, 64, 16, seed=6)
    cache, tables, lens, st = case.on_gpu()
    k = torch.zeros(case.T + 3, 2, 64, dtype=torch.float16, device="cuda")
    q = case.rows(2, tokens=case.T + 3)
    v = case.rows(2, tokens=case.T + 3)
    f, _ = freq(64)
    out = torch.full_like(q, 7.0)
    awq.cache_append(q, k, v, cache, tables, lens, st, inv_freq=f, out=out)
    assert bool((out[case.T:] == 7.0).all()) and not bool((out[:case.T] == 7.0).all(-1).any())
    kk, vv = (torch.full_like(v, 9.0) for _ in range(2))
    awq.cache_read(cache, tables, lens, st, tokens=case.T + 3, out=(kk, vv))
    assert bool((kk[case.T:] == 9.0).all()) and bool((kk[:4] == 0).all())      # a block of zeros: scale 0
    after = host_cache(cache)
    assert after[1][case.tables[0, 0]].max() == 0.0
    where = C.places(case.starts, case.lens, case.T)
    check_blocks(case.cache[2:], after[2:], R.to_f64(v)[:case.T], case, where)


def test_starts_that_make_no_sense(gpu):
    """Rows that descend or pass T are brought into bounds: nothing outside the call's arrays is touched."""
    import torch
    announce("append odd starts")
    case = Case([(4, 3), (5, 2), (6, 60)], 2, 2, 64, 16, seed=7)
    cache, tables, lens, _ = case.on_gpu()
    x = case.rows(2)
    f, _ = freq(64)
    for st in ([0, 9, 4, 15], [-5, 3, 99, 1 << 30], [15, 10, 5, 0], [7, 7, 7, 7]):
        out, raw, n = guarded_empty(tuple(x.shape), x.dtype)
        awq.cache_append(x, x, x, cache, tables, lens, ints(st), inv_freq=f, out=out)
        k, _ = awq.cache_read(cache, tables, lens, ints(st), tokens=case.T)
        torch.cuda.synchronize()
        assert sentinel_intact(raw, n)


def test_long_context_and_many_sequences(gpu):
    announce("append long")
    run(Case([(1, 70000), (700, 65000)], 2, 1, 64, 64, seed=8))
    run(Case([((b * 7) % 5, (b * 37) % 150) for b in range(200)], 2, 1, 64, 16, seed=9))
    run(Case([((b * 7) % 3, (b * 37) % 40) for b in range(5000)], 1, 1, 64, 16, seed=10))
    run(Case([(40 * (b % 2), (b * 37) % 40) for b in range(300)], 1, 1, 64, 16, seed=11))
    run(Case([(1, (b * 37) % 40) for b in range(9000)], 1, 1, 64, 32, seed=12), starts=False)
    # more rows than tokens, row by row and page by page
    run(Case([(5, 0), (3, 20), (40, 0)], 2, 2, 64, 16, seed=13, lens=[2, 23, 17]))
    run(Case([(90, 0), (3, 20), (60, 0)], 2, 2, 64, 16, seed=14, lens=[33, 23, 1]))


def test_refused(gpu):
    case = Case([(3, 4)], 4, 2, 64, 16)
    cache, tables, lens, st = case.on_gpu()
    q, k = case.rows(4), case.rows(2)
    f, _ = freq(64)
    ok = dict(q=q, k=k, v=k, cache=cache, tables=tables, lens=lens, starts=st, inv_freq=f)
    for bad in (dict(k=k.float()), dict(q=q.bfloat16()), dict(lens=lens.long()), dict(inv_freq=f.half())):
        with pytest.raises(TypeError):
            awq.cache_append(**{**ok, **bad})
    for bad in (dict(k=k[:2]), dict(v=k[:, :1]), dict(q=q[:2]), dict(cache=(cache[0], cache[1][:1], cache[2], cache[3])),
                dict(starts=st[:1]), dict(tables=tables[0]), dict(lens=lens.cpu()), dict(layout="x"), dict(out=q[:, :2])):
        with pytest.raises((ValueError, TypeError)):
            awq.cache_append(**{**ok, **bad})
    with pytest.raises(ValueError):
        awq.cache_read(cache, tables, lens, st)
    with pytest.raises(awq.AwqError):
        awq.cache_append(**{**ok, "starts": None})             # three rows, one sequence
