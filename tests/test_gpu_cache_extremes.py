"""Attention at the ends of what numbers hold."""
import numpy as np
import pytest

import weight_only_quantization_pack_amd as awq

import block_reference as R
from cache_util import Case, gpu as put, ints
from gpu_util import announce

pytestmark = pytest.mark.gpu

# rows a kv head: few, and many (tiles of 128 and 256)
SHAPES = [([(1, 300), (1, 77)], 4, 2, 64, 16), ([(1, 2100)], 8, 2, 128, 64), ([(40, 200)], 4, 2, 64, 16),
          ([(90, 300)], 4, 2, 128, 64), ([(70, 500)], 2, 1, 192, 128)]


def one_key(case, codes, size):
    """Queries of one channel, `size` by row and head, over keys of `codes`; the one key with the highest score takes all:
    (got, lse, the key's values, its score)."""
    import torch
    x = np.zeros((case.T, case.heads, case.dim), np.float32)
    x[..., 0] = size
    case.cache[1][:] = 1.0
    case.cache[3][:] = 2.0 ** -5                 # one value scale: its logarithm is rounded away beside such scores
    case.cache[0][..., 0] = codes
    q = put(x).to(case.dtype)
    lse = torch.zeros(case.T, case.heads, device="cuda")
    cache, tables, lens, st = case.on_gpu()
    got = awq.cache_attention(q, cache, tables, lens, st, scale=1.0, max_new=max(case.new), lse=lse)
    want, score = np.zeros(x.shape), np.zeros(x.shape[:2])
    q = R.to_f64(q)
    for b in range(len(case.lens)):
        for row in range(case.starts[b], case.starts[b + 1]):
            keys = np.arange(case.lens[b] - case.starts[b + 1] + row + 1)
            p, slot = case.tables[b, keys // case.page], keys % case.page
            for h in range(case.heads):
                g = h // (case.heads // case.kv)
                z = q[row, h, 0] * case.cache[0][p, g, slot, 0].astype(np.float64)
                best = np.flatnonzero(z == z.max())
                values = case.cache[2][p[best], g, slot[best]] * case.cache[3][p[best], g][:, None].astype(np.float64)
                want[row, h], score[row, h] = values.mean(0), z.max()
    return R.to_f64(got), R.to_f64(lse), want, score


def near(case, got, lse, want, score):
    """Keys of the highest score share it (their scores are the same numbers): a weight's and a scale's rounding, one to
    the type, and the bias of 128 in fp32 sums; the logarithm is the score's rounding and 2^-23 of it."""
    assert np.all(np.abs(got - want) <= 2.0 * R.unit(case.dtype) * np.abs(want) + (2.0 ** -11 + 2.0 ** -16) * 128.0 * 2.0 ** -5)
    assert np.all(np.abs(lse - score) <= 2.0 ** -21 * np.abs(score) + 12.0)


@pytest.mark.parametrize("exponent", [20, 24, 27, 30, 40, 70])
@pytest.mark.parametrize("pairs,heads,kv,dim,page", SHAPES, ids=str)
def test_large_scores(gpu, pairs, heads, kv, dim, page, exponent):
    """Scores of up to 2^77: the softmax is all one key's (or all of those that share its score)."""
    announce("attention large scores", pairs, heads, kv, dim, page, exponent)
    case = Case(pairs, heads, kv, dim, page, "bf16", seed=dim + exponent)
    g = np.random.default_rng(exponent)
    codes = g.integers(20, 128, case.cache[0].shape[:3])
    size = 2.0 ** exponent * (1.0 + g.integers(0, 100, (case.T, heads)) / 128.0)
    near(case, *one_key(case, codes, size))


@pytest.mark.parametrize("pairs,heads,kv,dim,page", SHAPES, ids=str)
def test_all_scores_far_below_zero(gpu, pairs, heads, kv, dim, page):
    """Every score below -2^98 * 50: the least of them takes all, and no row counts as one without keys."""
    announce("attention scores far below zero", pairs, heads, kv, dim, page)
    case = Case(pairs, heads, kv, dim, page, "bf16", seed=dim)
    g = np.random.default_rng(page)
    codes = g.integers(50, 128, case.cache[0].shape[:3])
    near(case, *one_key(case, codes, np.full((case.T, heads), -2.0 ** 98)))


def test_a_length_near_two_to_the_31(gpu):
    """2^31 - 1 tokens, all of them in one page: the first 32 tokens of each 128 say -100, the others 100, all with
    the same score.  A wave adds 2^15 steps in fp32, which round one way at worst: 2^-9 of (100 + the bias of 128)."""
    import torch
    announce("attention 2^31 - 1 tokens")
    page, dim, n = 128, 64, (1 << 31) - 1
    codes = torch.zeros(1, 1, page, dim, dtype=torch.int8, device="cuda")
    values = torch.full_like(codes, 100)
    values[:, :, :32] = -100
    one = torch.ones(1, 1, device="cuda")
    q = torch.randn(1, 1, dim, device="cuda").half()
    tables = torch.zeros(1, 1 << 24, dtype=torch.int32, device="cuda")
    lse = torch.zeros(1, 1, device="cuda")
    out = awq.cache_attention(q, (codes, one, values, one), tables, ints([n]), lse=lse)
    assert float((out.float() - 50.0).abs().max()) <= 2.0 ** -9 * 228 + 2.0 ** -11 * 50
    assert abs(float(lse) - np.log(n)) <= 2.0 ** -9


@pytest.mark.parametrize("window", [0, 200])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("pairs,heads,kv,dim,page", SHAPES + [([(130, 4000)], 4, 2, 64, 64), ([(200, 0), (90, 1500)], 2, 1, 128, 32)],
                         ids=str)
def test_large_scores_in_one_page(gpu, pairs, heads, kv, dim, page, sign, window):
    """One page's scores are 2^33 and more, or as far below zero, among ordinary ones: it takes all of every row that sees it,
    or nothing unless the row sees nothing else.  Its codes differ (but two of 128), so one of its
    tokens is the largest.  Ordinary scores are one product, right to 2^-22, so what is left is the weights' 2^-11 and what fp32 sums lose to the bias of 128."""
    announce("attention one large page", pairs, heads, kv, dim, page, sign, window)
    case = Case(pairs, heads, kv, dim, page, "bf16", seed=dim + page)
    g = np.random.default_rng(page + window)
    case.cache[0][..., 0] = g.integers(-127, 128, case.cache[0].shape[:3])
    case.cache[1][:], case.cache[3][:] = 2.0 ** -7, 2.0 ** -5
    for b, n in enumerate(case.lens):
        p = case.tables[b, (n - 1) // (2 * page)]
        case.cache[1][p] = 2.0 ** 33
        case.cache[0][p, :, :, 0] = sign * np.resize(1 + g.permutation(127), page)
    x = np.zeros((case.T, heads, dim), np.float32)
    x[..., 0] = 1.0 + g.integers(0, 128, (case.T, heads)) / 128.0
    q = put(x).to(case.dtype)
    cache, tables, lens, st = case.on_gpu()
    got = R.to_f64(awq.cache_attention(q, cache, tables, lens, st, scale=1.0, window=window, max_new=max(case.new)))
    x = R.to_f64(q)
    for b in range(len(case.lens)):
        for row in range(case.starts[b], case.starts[b + 1]):
            pos = case.lens[b] - case.starts[b + 1] + row
            keys = np.arange(max(0, pos - window + 1) if window else 0, pos + 1)
            p, slot = case.tables[b, keys // page], keys % page
            for h in range(heads):
                k = h // (heads // kv)
                z = x[row, h, 0] * case.cache[0][p, k, slot, 0] * case.cache[1][p, k].astype(np.float64)
                share = np.exp(z - z.max())
                v = case.cache[2][p, k, slot] * 2.0 ** -5
                want = share @ v / share.sum()
                size = share @ np.abs(v) / share.sum()
                assert np.all(np.abs(got[row, h] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * size + 2.0 ** -16 * 4.0), (row, h)
