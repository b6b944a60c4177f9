"""GPU parity of awq_cache_attention against 64 bits, within the bound that cache_reference.attention derives
for each output from the kernel's roundings."""
import math

import numpy as np
import pytest

import weight_only_quantization_pack_amd as awq

import block_reference as R
import cache_reference as C
from cache_util import DTYPES, Case, gpu as put, ints
from gpu_util import announce, guarded_empty, sentinel_intact

pytestmark = pytest.mark.gpu


def run(case, starts=True, window=0, softcap=0.0, scale=None, spread=2.5, max_new=None, max_len=None, q=None):
    import torch
    cache, tables, lens, st = case.on_gpu()
    q = case.rows(case.heads, spread) if q is None else q
    out, raw, n = guarded_empty((case.T, case.heads, case.dim), case.dtype)
    lse = torch.full((case.T, case.heads), 55.0, device="cuda")
    awq.cache_attention(q, cache, tables, lens, st if starts else None, scale=scale, window=window, softcap=softcap,
                        max_new=max_new, max_len=max_len, lse=lse, out=out)
    torch.cuda.synchronize()
    assert sentinel_intact(raw, n)
    ref, ref_lse, bound = C.attention(R.to_f64(q), case.cache, case.tables, case.lens, case.starts,
                                      case.dim ** -0.5 if scale is None else scale, window, softcap)
    got = R.to_f64(out)
    bound = bound + R.unit(out.dtype) * (np.abs(ref) + bound) + 2.0 ** -24
    # past the type's largest number (fp16: 65504, infinity from 65520 on) there is nothing to be near to
    top = torch.finfo(out.dtype).max
    fits = np.abs(ref) + bound < top
    assert np.all(np.isfinite(got[fits])) and np.all((np.abs(got) > 0.9 * top)[np.abs(ref) - bound > top])
    got, ref, bound = got[fits], ref[fits], bound[fits]
    worst = np.max(np.abs(got - ref) / bound) if got.size else 0.0
    assert worst <= 1.0, f"{worst:.3f} of the bound"
    lse = lse.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isneginf(lse), np.isneginf(ref_lse))
    some = np.isfinite(ref_lse)
    # scores as in the bound, and a logarithm
    assert np.all(np.abs(lse[some] - ref_lse[some]) <= 1e-3 + 2.0 ** -20 * np.abs(ref_lse[some]))
    return out


# lengths from one token to some thousands; empty sequences; ends inside pages and steps
DECODE = [[0], [1], [15], [31], [32], [100], [5, 0, 64, 63, 200, 1], [1000, 3], [4097]]


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("past", DECODE, ids=str)
def test_decode(gpu, past, page):
    announce("attention decode", past, page)
    run(Case([(1, n) for n in past], 8, 2, 128, page, seed=sum(past) + page), starts=False)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 3), (8, 1), (10, 2), (32, 1), (48, 2), (80, 1)])
def test_heads_and_types(gpu, heads, kv, dim, dtype):
    announce("attention heads", heads, kv, dim, dtype)
    for page in (16, 32, 128):
        run(Case([(1, 70), (1, 0), (1, 333)], heads, kv, dim, page, dtype, seed=heads + dim + page))


ROWS = [[(2, 0)], [(5, 60)], [(3, 5), (8, 300), (1, 31), (0, 9), (16, 0)], [(33, 0)], [(70, 129)], [(130, 3), (1, 500)],
        [(300, 0), (17, 1000)], [(259, 40)]]


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("heads,kv,dim", [(4, 4, 64), (8, 2, 128), (5, 1, 96), (6, 2, 256)])
@pytest.mark.parametrize("pairs", ROWS, ids=str)
def test_several_rows(gpu, pairs, heads, kv, dim, page):
    announce("attention rows", pairs, heads, kv, dim, page)
    run(Case(pairs, heads, kv, dim, page, "bf16" if dim == 256 else "fp16", seed=len(pairs) + dim + page))


@pytest.mark.parametrize("window", [1, 7, 32, 100, 5000])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_window_and_cap(gpu, window, softcap):
    announce("attention window", window, softcap)
    for page in (16, 64):
        run(Case([(1, 0), (1, 299), (1, 64)], 8, 2, 128, page, seed=window), window=window, softcap=softcap)
        run(Case([(40, 3), (2, 257), (90, 200)], 4, 2, 64, page, "bf16", seed=window + 1), window=window, softcap=softcap)


def test_rows_without_keys(gpu):
    """More rows than tokens, no tokens at all, pages outside the cache, tables that end early: 0 and -infinity."""
    announce("attention empty rows")
    case = Case([(6, 0), (4, 0), (5, 20)], 4, 2, 64, 16, seed=1, lens=[2, 0, 25])
    out = run(case)
    assert not bool(out[:4].any()) and not bool(out[6:10].any())
    run(Case([(20, 40), (1, 200)], 4, 2, 64, 16, seed=2, bad=[(0, 0, -1), (0, 2, 10 ** 9), (1, 5, -7), (1, 12, 1 << 30)]))
    run(Case([(20, 40), (1, 200)], 4, 2, 64, 64, seed=3, bad=[(0, 0, -1), (1, 1, 10 ** 9), (1, 3, -2)]))
    run(Case([(1, 0)], 4, 2, 64, 32, seed=4, bad=[(0, 0, -1)]), starts=False)
    run(Case([(5, 90), (1, 40)], 4, 2, 128, 32, seed=5, lens=[130, 41]))          # tokens past the table


def test_scales_far_apart(gpu):
    """Blocks whose scales differ by powers of ten, blocks of zeros with scale 0."""
    announce("attention scales")
    for dim, page in ((128, 16), (64, 64)):
        case = Case([(1, 500), (30, 200)], 4, 2, dim, page, seed=6)
        case.cache[3] = (case.cache[3] * 10.0 ** case.g.uniform(-6, 6, case.cache[3].shape)).astype(np.float32)
        zero = case.g.random(case.cache[3].shape) < 0.3
        case.cache[3][zero] = 0.0
        case.cache[2][zero] = 0
        case.cache[1][case.g.random(zero.shape) < 0.2] = 0.0
        run(case)
        run(case, spread=1e-3)


def test_large_and_small_queries(gpu):
    announce("attention query sizes")
    run(Case([(1, 300), (9, 40)], 4, 2, 128, 64, seed=7), spread=1e-4)
    run(Case([(1, 300), (9, 40)], 4, 2, 128, 64, "bf16", seed=8), spread=1e-20)
    run(Case([(1, 300), (9, 40)], 4, 2, 128, 64, "bf16", seed=9), spread=1e20, scale=1e-20)
    case = Case([(1, 300), (9, 40)], 4, 2, 128, 64, seed=10)
    run(case, q=case.rows(4) * 0)
    run(case, scale=0.0)
    run(case, scale=-0.1)


def test_other_bounds_than_the_lengths(gpu):
    """max_new and max_len choose kernels; the results hold for longer sequences too."""
    announce("attention bounds")
    for pairs in ([(1, 700), (1, 90)], [(40, 500), (3, 2)]):
        for new, most in ((1, 1), (1, 100000), (64, 64), (100000, 100000)):
            run(Case(pairs, 8, 2, 128, 32, seed=11), max_new=new, max_len=most)


def test_strides_rows_behind_and_other_stream(gpu):
    import torch
    announce("attention strides")
    case = Case([(3, 100), (20, 9)], 6, 2, 128, 64, seed=12)
    cache, tables, lens, st = case.on_gpu()
    qkv = case.rows(10, 2.0, tokens=case.T + 5)
    q = qkv[:, 2:8]
    want = awq.cache_attention(q[:case.T].contiguous(), cache, tables, lens, st)
    out = torch.full((case.T + 5, 6, 128), 7.0, dtype=case.dtype, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        awq.cache_attention(q, cache, tables, lens, st, out=out)
    stream.synchronize()
    assert torch.equal(out[:case.T], want) and bool((out[case.T:] == 7.0).all())


def test_starts_that_make_no_sense(gpu):
    import torch
    announce("attention odd starts")
    case = Case([(4, 3), (5, 2), (6, 600)], 4, 2, 64, 16, seed=13)
    cache, tables, lens, _ = case.on_gpu()
    q = case.rows(4)
    for st in ([0, 9, 4, 15], [-5, 3, 99, 1 << 30], [15, 10, 5, 0], [7, 7, 7, 7]):
        for most in (64, 100000):
            out, raw, n = guarded_empty(tuple(q.shape), q.dtype)
            awq.cache_attention(q, cache, tables, lens, ints(st), out=out, max_len=most)
            torch.cuda.synchronize()
            assert sentinel_intact(raw, n)


@pytest.mark.parametrize("new,dim", [(1, 128), (4, 128), (200, 128), (20, 256), (200, 256), (200, 192)])
def test_two_graphs_share_a_workspace(gpu, new, dim):
    """Captured calls on one workspace full of something else, replayed in turns with eager work between."""
    import torch
    announce("attention graphs", new, dim)
    calls = []
    for seed in (14, 15):
        case = Case([(new, 900 + 50 * seed), (new, 31), (new, 0)], 8, 2, dim, 64, seed=seed)
        calls.append((case, case.rows(8, 2.0), *case.on_gpu()))
    sizes = [awq.cache_attention_workspace_bytes(3 * new, 3, 8, 2, dim, new, c[3].shape[1] * 64) for c in calls]
    ws = torch.full((max(sizes) + 16,), 0xFF, dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(c[1]) for c in calls]

    def go(i):
        _, q, cache, tables, lens, st = calls[i]
        awq.cache_attention(q, cache, tables, lens, st, max_new=new, out=outs[i], workspace=ws)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs = [torch.cuda.CUDAGraph() for _ in calls]
    with torch.cuda.stream(stream):
        go(0)
        go(1)
    stream.synchronize()
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g, stream=stream):
            go(i)
    for turn in range(3):
        for i in (0, 1):
            calls[i][1].copy_(calls[i][0].rows(8, 2.0))
            ws.fill_(turn)
            outs[i].zero_()
            torch.cuda.synchronize()
            graphs[i].replay()
            torch.cuda.synchronize()
            got = outs[i].clone()
            go(i)
            torch.cuda.synchronize()
            assert torch.equal(got, outs[i])


def test_many_ragged_sequences(gpu):
    announce("attention ragged")
    run(Case([((b * 5) % 4, (b * 61) % 400) for b in range(150)], 4, 1, 64, 32, seed=16))
    run(Case([(1, (b * 131) % 900) for b in range(90)], 8, 2, 128, 64, "bf16", seed=17), starts=False)


def test_thousands_of_sequences(gpu):
    """Sequences found by more than one look at the starts; most of them short, some without rows."""
    announce("attention thousands")
    for new, most in ((1, 60), (2, 60), (1, 4000), (3, 4000)):
        pairs = [((b * 7) % (new + 1), (b * 13) % 50) for b in range(4500)]
        run(Case(pairs, 2, 1, 64, 16, seed=new + most), max_new=new, max_len=most)
    pairs = [((b * 7) % 5, (b * 13) % 50) for b in range(700)]
    run(Case(pairs, 20, 1, 64, 16, seed=21), max_new=4)


def test_one_long_sequence(gpu):
    announce("attention long")
    run(Case([(1, 30000)], 8, 2, 128, 64, seed=18), starts=False)
    run(Case([(3, 9000)], 4, 1, 128, 16, "bf16", seed=19))


def test_blocks_past_four_gigabytes(gpu):
    """Pages whose codes start beyond 2^32 bytes."""
    import torch
    announce("attention past 4 GB")
    kv, page, dim = 8, 128, 128
    pages = (1 << 32) // (kv * page * dim) + 40
    case = Case([(1, 200), (5, 300)], 16, kv, dim, page, seed=20)
    small, _, lens, st = case.on_gpu()
    big = [torch.zeros((pages, *c.shape[1:]), dtype=c.dtype, device="cuda") for c in small]
    place = torch.arange(case.pages, device="cuda") * 0 + torch.arange(case.pages, device="cuda").flip(0) + pages - case.pages
    for a, b in zip(big, small):
        a[place] = b
    tables = np.where(case.tables >= 0, place.cpu().numpy()[np.maximum(case.tables, 0)], -1).astype(np.int32)
    q = case.rows(16)
    want = awq.cache_attention(q, small, put(case.tables), lens, st)
    assert torch.equal(awq.cache_attention(q, big, put(tables), lens, st), want)
    k, v = awq.cache_read(big, put(tables), lens, st, tokens=case.T)
    k2, v2 = awq.cache_read(small, put(case.tables), lens, st, tokens=case.T)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    x = case.rows(kv)
    for cache, t in ((big, put(tables)), (small, put(case.tables))):
        awq.cache_append(None, x, x, cache, t, lens, st)
    for a, b in zip(big, small):
        assert torch.equal(a[place], b)


def test_refused(gpu):
    import torch
    case = Case([(3, 400)], 4, 2, 64, 16)
    cache, tables, lens, st = case.on_gpu()
    q = case.rows(4)
    ok = dict(q=q, cache=cache, tables=tables, lens=lens, starts=st)
    for bad in (dict(q=q.float()), dict(lens=lens.long()), dict(cache=(cache[0].float(), *cache[1:]))):
        with pytest.raises(TypeError):
            awq.cache_attention(**{**ok, **bad})
    for bad in (dict(q=q[0]), dict(q=q[..., :32]), dict(starts=st[:1]), dict(tables=tables[0]), dict(lse=torch.zeros(3, 4)),
                dict(out=q[:2]), dict(workspace=torch.zeros(4, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            awq.cache_attention(**{**ok, **bad})
    for bad in (dict(q=q[:, :3].contiguous()), dict(window=-1), dict(softcap=-1.0), dict(scale=math.nan), dict(max_new=0),
                dict(starts=None), dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(awq.AwqError):
            awq.cache_attention(**{**ok, **bad})


@pytest.mark.parametrize("softcap", [2.0 ** -10, 0.5, 1024.0])
def test_ends_of_the_caps(gpu, softcap):
    announce("attention caps", softcap)
    run(Case([(1, 77), (1, 700)], 4, 2, 64, 16, seed=61), softcap=softcap)
    run(Case([(150, 20)], 4, 2, 64, 16, seed=62), softcap=softcap)


@pytest.mark.parametrize("heads,kv", [(71, 1), (128, 1), (200, 2), (300, 1)])
def test_many_heads_share_one(gpu, heads, kv):
    """More rows than a tile's from single tokens."""
    announce("attention shared heads", heads, kv)
    for dim in (64, 192):
        run(Case([(1, 400), (1, 0), (1, 2050)], heads, kv, dim, 32, seed=heads + dim), starts=False)
    run(Case([(2, 90), (0, 3), (3, 0)], heads, kv, 128, 16, "bf16", seed=heads))


@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("pairs,heads,kv,dim,page", [([(130, 6000)], 4, 2, 64, 64), ([(100, 5000), (100, 0), (64, 700)], 4, 1, 128, 16),
                                                     ([(90, 4000), (0, 50), (200, 10)], 2, 2, 192, 32),
                                                     ([(70, 9000), (1, 40)], 8, 1, 96, 128)], ids=str)
def test_tiles_of_different_parts(gpu, pairs, heads, kv, dim, page, window):
    """Long tiles in parts beside short ones in fewer or one; also with bounds that are smaller than the lengths."""
    announce("attention parts", pairs, heads, kv, dim, page, window)
    most = max(n + p for n, p in pairs)
    need = awq.cache_attention_workspace_bytes(sum(n for n, _ in pairs), len(pairs), heads, kv, dim,
                                               max(n for n, _ in pairs), most)
    assert need > 0
    run(Case(pairs, heads, kv, dim, page, seed=dim), window=window, max_new=max(n for n, _ in pairs), max_len=most)
    run(Case(pairs, heads, kv, dim, page, "bf16", seed=dim + 1), window=window, max_new=40, max_len=most // 2)
