"""The cache's book on the GPU against lists: whole numbers, so everything is equal."""
import numpy as np
import pytest

import weight_only_quantization_pack_amd as awq

import cache_reference as C
from cache_util import gpu as put, ints
from gpu_util import announce

pytestmark = pytest.mark.gpu


class Pair:
    """A book on the GPU and the same in lists."""

    def __init__(self, rows, lens, pages, page, width, extra=()):
        refs = [0] * pages
        for r in rows:
            for p in r:
                refs[p] += 1
        for p in extra:                                   # pages that the caller keeps
            refs[p] += 1
        self.page, self.width = page, width
        self.list = C.Book(rows, lens, refs, page)
        self.tables, self.lens, self.refs = ints(self.list.table(width)).reshape(-1, width), ints(lens), ints(refs)

    def check(self):
        assert self.tables.cpu().tolist() == self.list.table(self.width)
        assert self.lens.cpu().tolist() == self.list.lens
        assert self.refs.cpu().tolist() == self.list.refs

    def fork(self, parents):
        self.list.fork(parents)
        self.tables, self.lens = awq.cache_fork(self.tables, self.lens, self.refs, ints(parents), self.page)
        self.check()

    def reserve(self, counts):
        pairs, status = self.list.reserve(counts, self.width)
        got, st = awq.cache_reserve(self.tables, self.lens, self.refs, ints(counts), self.page)
        assert st.cpu().tolist() == status and got.cpu().tolist() == [list(p) for p in pairs]
        self.check()
        return pairs, status

    def compact(self):
        moves = self.list.compact()
        got, count = awq.cache_compact(self.tables, self.lens, self.refs, self.page)
        assert count.cpu().tolist() == [len(moves)]
        assert got.cpu().tolist() == [list(m) for m in moves] + [[-1, -1]] * (len(self.list.refs) - len(moves))
        self.check()
        return moves


def scattered(g, lens, pages, page):
    ids, at, rows = g.permutation(pages).tolist(), 0, []
    for n in lens:
        k = -(-n // page)
        rows.append(ids[at:at + k])
        at += k
    return rows


@pytest.mark.parametrize("seed", range(6))
def test_a_life_of_a_book(gpu, seed):
    """Rows forked, dropped, grown and compacted at random, page sizes and widths of all kinds."""
    announce("book", seed)
    g = np.random.default_rng(seed)
    page, pages, width = [16, 32, 64, 128][seed % 4], [70, 200, 1500, 33][seed % 4], [9, 40, 3, 300][seed % 4]
    lens = [int(v) for v in g.integers(0, min(width, 4) * page + 1, 6)]
    book = Pair(scattered(g, lens, pages, page), lens, pages, page, width, extra=[pages - 1] if seed % 2 else [])
    short = 0
    for _ in range(25):
        what = g.integers(0, 4)
        B = len(book.list.rows)
        if what == 0:
            n = int(g.integers(1, 12))
            book.fork([int(v) for v in g.integers(-1, B + (seed == 5), n)])
        elif what < 3:
            most = 1 if what == 1 else 2 * page
            _, status = book.reserve([int(v) for v in g.integers(-1, most + 1, B)])
            short += any(status)
        else:
            book.compact()
            used = sum(r > 0 for r in book.list.refs)
            assert all(r > 0 for r in book.list.refs[:used])


def test_shared_pages(gpu):
    """Who copies: all writers of a page that others keep; all but the first where they are its only holders."""
    announce("book shared")
    for extra, parents, counts in (((), [0, 0, 0], [1, 1, 1]), ((), [0, 0, 0], [0, 1, 1]), ((), [0, 0, 0], [1, 0, 0]),
                                   ([5], [0, 0, 0], [1, 1, 1]), ((), [0, 0, -1], [20, 33, 0]), ((), [0], [1])):
        book = Pair([[3, 5]], [20], 12, 16, 6, extra)
        book.fork(parents)
        pairs, status = book.reserve(counts)
        assert status == [0, 0]
    book = Pair([[3, 5]], [32], 12, 16, 6)                # a full last page is not written: nobody copies
    book.fork([0, 0])
    pairs, _ = book.reserve([1, 1])
    assert pairs == [(-1, -1)] * 2


def test_nothing_changes_when_it_does_not_fit(gpu):
    announce("book full")
    book = Pair([[0, 1], [2]], [20, 3], 5, 16, 3)
    assert book.reserve([30, 30])[1] == [0, 1]            # the first row would need a fourth page; the second fits
    assert book.reserve([28, 30])[1] == [1, 0]
    assert book.reserve([28, 13])[1] == [0, 0]
    assert book.reserve([1, 0])[1] == [0, 1]
    assert book.reserve([0, 20])[1] == [1, 0]
    assert book.reserve([0, (1 << 31) - 1])[1] == [0, 1]
    assert book.reserve([0, 0])[1] == [0, 0]


def test_many_rows_and_pages(gpu):
    announce("book large")
    g = np.random.default_rng(1)
    lens = [int(v) for v in g.integers(0, 300, 4096)]
    book = Pair(scattered(g, lens, 50000, 16), lens, 50000, 16, 20)
    book.reserve([int(v) for v in g.integers(0, 20, 4096)])
    book.fork([int(v) for v in g.integers(-1, 4096, 3000)])
    book.reserve([1] * 3000)
    book.compact()
    book = Pair([[70000, 5, 16383, 16384, 16385, 99999]], [96], 100000, 16, 20000)
    book.reserve([300000])
    book.compact()


def test_beams_of_one_prompt(gpu):
    """One row into many, and a batch that shrinks and grows."""
    announce("book beams")
    book = Pair([[7, 2, 9]], [40], 600, 16, 8)
    for parents, counts in (([0] * 300, [1] * 300), (list(range(299, -1, -1)), [1] * 300), ([5, 5, -1, 299], [50, 1, 1, 0]), ([-1], [0]),
                            ([-1, 0], [16, 17])):
        book.fork(parents)
        book.reserve(counts)


@pytest.mark.parametrize("layers", [None, 1, 3])
def test_copy_pages(gpu, layers):
    import torch
    announce("copy pages", layers)
    g = torch.Generator().manual_seed(0)
    lead = (40,) if layers is None else (layers, 40)
    # a unit, several, an odd number of words, one word, 16-bit elements
    shapes = [(8, 64, 128), (3, 16, 96), (3, 7), (1,), (20001,), (2, 5)]
    tensors = [torch.randint(-100, 100, (*lead, *s), generator=g).to(torch.int8 if i < 2 else torch.float32 if i < 5 else torch.float16).cuda()
               for i, s in enumerate(shapes)]
    for pairs, count in ([[(3, 9), (-1, -1), (0, 39), (39 * 0 + 3, 17), (5, 40), (41, 6), (38, 1)], None], [[(1, 2), (3, 4), (5, 6), (7, 8)], 2],
                         [[(1, 2)], 0], [[(1, 2), (3, 4)], 99], [[(1, 2)], -5], [[], None]):
        want = [t.clone() for t in tensors]
        n = len(pairs) if count is None else min(max(count, 0), len(pairs))
        for src, dst in pairs[:n]:
            if 0 <= src < 40 and 0 <= dst < 40:
                for t in want:
                    (t if layers is None else t.transpose(0, 1))[dst] = (t if layers is None else t.transpose(0, 1))[src].clone()
        awq.cache_copy_pages(tensors, ints(pairs).reshape(-1, 2), count=None if count is None else ints([count]), layers=layers)
        for a, b in zip(tensors, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("n,share", [(70, 0.5), (256, 1.0), (300, 0.3), (1000, 0.1), (4000, 0.9), (4096, 0.5), (4100, 0.2)])
def test_copy_of_long_lists(gpu, n, share):
    """Every valid pair of a list is copied, by many workgroups, wherever it stands."""
    import torch
    announce("copy long list", n, share)
    g = np.random.default_rng(n)
    pages = 2 * n + 10
    t = [torch.randint(-100, 100, (3, pages, k), dtype=torch.int8, device="cuda") for k in (64, 12)]
    order = g.permutation(pages)
    pairs = np.where(g.random(n)[:, None] < share, np.stack([order[:n], order[n:2 * n]], 1), -1).astype(np.int32)
    want = [a.clone() for a in t]
    some = pairs[pairs[:, 0] >= 0]
    for a in want:
        a[:, put(some[:, 1].copy()).long()] = a[:, put(some[:, 0].copy()).long()]
    awq.cache_copy_pages(t, put(pairs), layers=3)
    for a, b in zip(t, want):
        assert torch.equal(a, b)


def test_copy_past_four_gigabytes(gpu):
    import torch
    announce("copy past 4 GB")
    t = torch.zeros(2, 1100, 1 << 21, dtype=torch.uint8, device="cuda")
    t[1, 1099] = torch.arange(1 << 21, device="cuda").to(torch.uint8)
    t[0, 1099] = 3
    awq.cache_copy_pages([t], ints([(1099, 1)]), layers=2)
    assert torch.equal(t[1, 1], t[1, 1099]) and bool((t[0, 1] == 3).all()) and not bool(t[:, 0].any()) and not bool(t[:, 2].any())


def test_graph_of_a_step(gpu):
    """fork, reserve and the copies in a captured graph, replayed on other books."""
    import torch
    announce("book graph")
    g = np.random.default_rng(2)
    page, pages, width, B = 16, 120, 6, 6
    cache = awq.empty_cache(pages, 2, page, 64)
    cache[0].copy_(torch.randint(-127, 128, cache[0].shape, dtype=torch.int8, device="cuda"))
    first = [int(v) for v in g.integers(1, 60, B)]
    start = Pair(scattered(g, first, pages, page), first, pages, page, width)
    tables, lens, refs = start.tables.clone(), start.lens.clone(), start.refs.clone()
    parents, counts = ints([0] * B), ints([1] * B)
    out = torch.empty_like(tables), torch.empty_like(lens)
    pairs, status, moves, count = ints([[0, 0]] * B), ints([0, 0]), ints([[0, 0]] * pages), ints([0])

    def step():
        awq.cache_fork(tables, lens, refs, parents, page, out=out)
        awq.cache_reserve(*out, refs, counts, page, out=(pairs, status))
        awq.cache_copy_pages(cache, pairs)
        awq.cache_compact(*out, refs, page, out=(moves, count))
        awq.cache_copy_pages(cache, moves, count=count)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for turn in range(4):
        rows = [int(v) for v in g.integers(1, 60, B)]
        book = Pair(scattered(g, rows, pages, page), rows, pages, page, width)
        p = [int(v) for v in g.integers(-1, B, B)]
        tables.copy_(book.tables)
        lens.copy_(book.lens)
        refs.copy_(book.refs)
        parents.copy_(ints(p))
        want = cache[0].cpu().numpy().copy()
        graph.replay()
        torch.cuda.synchronize()
        book.list.fork(p)
        todo, state = book.list.reserve([1] * B, width)
        assert state == [0, 0] == status.cpu().tolist()
        for src, dst in [t for t in todo if t[0] >= 0] + book.list.compact():
            want[dst] = want[src]
        assert out[0].cpu().tolist() == book.list.table(width) and refs.cpu().tolist() == book.list.refs
        assert np.array_equal(cache[0].cpu().numpy(), want)


def test_refused(gpu):
    import torch
    t, l, r = ints([[0, -1]]), ints([5]), ints([1, 0, 0])
    with pytest.raises(TypeError):
        awq.cache_fork(t, l.long(), r, ints([0]), 16)
    for bad in (lambda: awq.cache_fork(t[0], l, r, ints([0]), 16), lambda: awq.cache_reserve(t, l, r, ints([1, 1]), 16),
                lambda: awq.cache_compact(t, ints([5, 5]), r, 16), lambda: awq.cache_copy_pages([], ints([[0, 1]])),
                lambda: awq.cache_copy_pages([torch.zeros(3, 4, device="cuda"), torch.zeros(4, 4, device="cuda")], ints([[0, 1]])),
                lambda: awq.cache_copy_pages([torch.zeros(3, 4, device="cuda")], ints([0, 1]))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: awq.cache_fork(t, l, r, ints([0]), 20), lambda: awq.cache_fork(t, l, r, ints([0]), 16, out=(t, ints([0]))),
                lambda: awq.cache_copy_pages([torch.zeros(3, 3, dtype=torch.int8, device="cuda")], ints([[0, 1]]))):
        with pytest.raises(awq.AwqError):
            bad()
    assert t.cpu().tolist() == [[0, -1]] and r.cpu().tolist() == [1, 0, 0]
