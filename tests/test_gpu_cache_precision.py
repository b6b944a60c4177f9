"""How near cache_attention comes to 64 bits, channel by channel and for the logarithm, within the bounds that
cache_bounds.attention counts."""
import numpy as np
import pytest

import weight_only_quantization_pack_amd as awq

import block_reference as R
import cache_bounds as Bounds
from cache_util import Case, gpu as put
from gpu_util import announce

pytestmark = pytest.mark.gpu

# three of few rows a kv head (up to 64: the cache goes straight into registers), three of many (tiles of 128 and 256)
SHAPES = [([(1, 300), (1, 77)], 4, 2, 64, 16), ([(1, 2100)], 8, 2, 128, 64), ([(5, 90)], 4, 1, 256, 32),
          ([(40, 200)], 4, 2, 64, 16), ([(90, 300)], 4, 2, 128, 64), ([(70, 500)], 2, 1, 192, 128)]


def check(case, spread=2.5, q=None, **kw):
    import torch
    cache, tables, lens, st = case.on_gpu()
    q = case.rows(case.heads, spread) if q is None else q
    lse = torch.full((case.T, case.heads), 55.0, device="cuda")
    scale = kw.get("scale", case.dim ** -0.5)
    got = awq.cache_attention(q, cache, tables, lens, st, max_new=max(case.new), lse=lse, **kw)
    few = max(case.new) * case.heads // case.kv <= 64
    ref, ref_lse, bound, lse_bound = Bounds.attention(R.to_f64(q), case.cache, case.tables, case.lens, case.starts, scale,
                                                      kw.get("window", 0), kw.get("softcap", 0.0), 128.0 if few else 0.0)
    bound = bound + R.unit(got.dtype) * (np.abs(ref) + bound) + 2.0 ** -24
    worst = np.max(np.abs(R.to_f64(got) - ref) / bound)
    assert worst <= 1.0, f"out: {worst:.3f} of the bound"
    lse = R.to_f64(lse)
    none = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(lse), none)
    worst = np.max(np.abs(lse[~none] - ref_lse[~none]) / lse_bound[~none], initial=0.0)
    assert worst <= 1.0, f"lse: {worst:.3f} of the bound"


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("pairs,heads,kv,dim,page", SHAPES, ids=str)
def test_channels_and_logarithms(gpu, pairs, heads, kv, dim, page, dtype):
    announce("attention precision", pairs, heads, kv, dim, page, dtype)
    for kw in (dict(), dict(window=60), dict(softcap=20.0)):
        check(Case(pairs, heads, kv, dim, page, dtype, seed=dim + page), **kw)


@pytest.mark.parametrize("far", [2.0 ** 10, 2.0 ** 18, 2.0 ** 26])
@pytest.mark.parametrize("pairs,heads,kv,dim,page", SHAPES, ids=str)
def test_one_page_with_a_large_channel(gpu, pairs, heads, kv, dim, page, far):
    """Values of one page are larger than all others, in one channel: the other channels get what they have from weights
    that are small beside that page's."""
    announce("attention large channel", pairs, heads, kv, dim, page, far)
    case = Case(pairs, heads, kv, dim, page, "bf16", seed=dim + page)
    case.cache[2][:] = 64 + np.abs(case.cache[2]) // 2          # of one sign: nothing cancels
    for b in range(len(pairs)):
        p = case.tables[b, 1 if pairs[b][1] > page else 0]
        case.cache[2][p, ..., 1:] = 0
        case.cache[3][p] *= far
    check(case)


@pytest.mark.parametrize("pairs,heads,kv,dim,page", SHAPES, ids=str)
def test_a_key_that_takes_nearly_all(gpu, pairs, heads, kv, dim, page):
    """The first token has most of the softmax and values of zero: the output is the tail's."""
    announce("attention tail", pairs, heads, kv, dim, page)
    for nats in (11.0, 15.0, 19.0):
        case = Case(pairs, heads, kv, dim, page, "bf16", seed=dim + page + 1)
        g = np.random.default_rng(7)
        x = np.zeros((case.T, case.heads, case.dim), np.float32)
        x[..., 0] = nats * case.dim ** 0.5       # the only channel of the queries; its keys are 1 for the first token
        case.cache[2][:] = 64 + np.abs(case.cache[2]) // 2      # of one sign: nothing cancels
        case.cache[1][:] = 2.0 ** -6
        case.cache[0][..., 0] = g.integers(-4, 5, case.cache[0].shape[:3])
        for b in range(len(pairs)):
            case.cache[0][case.tables[b, 0], :, 0, 0] = 64
            case.cache[2][case.tables[b, 0], :, 0] = 0
        check(case, q=put(x).to(case.dtype))
