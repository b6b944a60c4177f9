"""The cache's operators as a decode step uses them: reserve, copy, append, attend and
fork on one book, against the same steps in lists and 64 bits; eagerly, in a graph,
and on two streams at once."""
import numpy as np
import pytest

import weight_only_quantization_pack_amd as awq

import block_reference as R
import cache_reference as C
from cache_util import DTYPES, dtype_of, freq, gpu as put, host_cache, ints
from gpu_util import announce

pytestmark = pytest.mark.gpu


class Step:
    """Buffers of a decode step of B sequences, as a graph would hold them."""

    def __init__(self, B, kv, group, dim, page, pages, width, dtype, seed):
        import torch
        g = np.random.default_rng(seed)
        self.B, self.kv, self.h, self.dim, self.page, self.width = B, kv, kv * group, dim, page, width
        lens = g.integers(1, (width - 1) * page, B)
        ids, at, rows = g.permutation(pages).tolist(), 0, []
        for n in lens:
            k = -(-int(n) // page)
            rows.append(ids[at:at + k])
            at += k
        refs = [0] * pages
        for r in rows:
            for p in r:
                refs[p] += 1
        self.book = C.Book(rows, [int(n) for n in lens], refs, page)
        self.tables, self.lens, self.refs = ints(self.book.table(width)), ints(self.book.lens), ints(refs)
        self.next = torch.empty_like(self.tables), torch.empty_like(self.lens)
        self.cache = awq.empty_cache(pages, kv, page, dim)
        for i in (0, 2):
            self.cache[i].copy_(put(np.clip(np.rint(32 * g.standard_normal(self.cache[i].shape)), -127, 127).astype(np.int8)))
            self.cache[i + 1].copy_(put((0.03 * np.exp(0.3 * g.standard_normal(self.cache[i + 1].shape))).astype(np.float32)))
        self.qkv = torch.zeros(B, self.h + 2 * kv, dim, dtype=dtype_of(dtype), device="cuda")
        self.parents, self.counts = ints(list(range(B))), ints([1] * B)
        self.pairs, self.status = ints([[0, 0]] * B), ints([0, 0])
        self.turned, self.out = (torch.zeros(B, self.h, dim, dtype=self.qkv.dtype, device="cuda") for _ in range(2))
        self.f, _ = freq(dim)
        self.ws = torch.empty(awq.cache_attention_workspace_bytes(B, B, self.h, kv, dim, 1, width * page) + 16,
                              dtype=torch.uint8, device="cuda")
        self.g = g

    def fill(self, parents):
        x = self.g.standard_normal(tuple(self.qkv.shape)).astype(np.float32)
        self.qkv.copy_(put(x).to(self.qkv.dtype))
        self.parents.copy_(ints(parents))

    def run(self):
        """Rows from their parents, room, copies, the new token in, attention."""
        h, kv = self.h, self.kv
        awq.cache_fork(self.tables, self.lens, self.refs, self.parents, self.page, out=self.next)
        awq.cache_reserve(*self.next, self.refs, self.counts, self.page, out=(self.pairs, self.status))
        awq.cache_copy_pages(self.cache, self.pairs)
        tables, lens = self.next
        awq.cache_append(self.qkv[:, :h], self.qkv[:, h:h + kv], self.qkv[:, h + kv:], self.cache, tables, lens,
                         inv_freq=self.f, out=self.turned)
        awq.cache_attention(self.turned, self.cache, tables, lens, out=self.out, workspace=self.ws)
        self.tables.copy_(tables)
        self.lens.copy_(lens)

    def check(self, before, parents):
        """The step that was just run, from the cache as it was before."""
        self.book.fork(parents)
        pairs, status = self.book.reserve([1] * self.B, self.width)
        assert status == [0, 0] == self.status.cpu().tolist()
        assert self.tables.cpu().tolist() == self.book.table(self.width)
        assert self.lens.cpu().tolist() == self.book.lens and self.refs.cpu().tolist() == self.book.refs
        for src, dst in pairs:
            if src >= 0:
                for t in before:
                    t[dst] = t[src]
        tables, lens = np.array(self.book.table(self.width)), self.book.lens
        starts = list(range(self.B + 1))
        where = C.places(starts, lens, self.B)
        pos = np.array([p for _, p in where])
        qkv, f = R.to_f64(self.qkv), self.f.cpu().numpy()
        turned = C.rope(qkv[:, :self.h + self.kv], pos, f)
        after = host_cache(self.cache)
        for x, i in ((turned[:, self.h:], 0), (qkv[:, self.h + self.kv:], 2)):
            for (p, head), (scale, slots) in C.append(x, before[i], before[i + 1], tables, where, self.page).items():
                assert abs(after[i + 1][p, head] - scale) <= 2.0 ** -19 * scale
                for s, exact in slots.items():
                    assert np.abs(after[i][p, head, s] - exact).max() <= 0.5 + 127 * 2.0 ** -18
        ref, _, bound = C.attention(R.to_f64(self.turned), after, tables, lens, starts, self.dim ** -0.5)
        bound = bound + R.unit(self.out.dtype) * (np.abs(ref) + bound) + 2.0 ** -24
        worst = np.max(np.abs(R.to_f64(self.out) - ref) / bound)
        assert worst <= 1.0, f"{worst:.3f} of the bound"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,kv,group,dim,page", [(1, 2, 4, 128, 16), (6, 2, 2, 64, 32), (12, 1, 5, 96, 16), (5, 3, 1, 256, 64)])
def test_decode_steps(gpu, B, kv, group, dim, page, dtype):
    announce("cache together", B, kv, group, dim, page, dtype)
    s = Step(B, kv, group, dim, page, 60 * B, 6, dtype, seed=B)
    for step in range(5):
        parents = [int(p) for p in s.g.integers(0, B, B)]
        s.fill(parents)
        before = host_cache(s.cache)
        s.run()
        if int(s.status.sum()):
            break
        s.check(before, parents)


def test_decode_steps_in_a_graph(gpu):
    import torch
    announce("cache together, graph")
    s = Step(6, 2, 4, 128, 16, 400, 8, "bf16", seed=3)
    start = [t.clone() for t in (s.tables, s.lens, s.refs, *s.cache)]
    s.fill(list(range(6)))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        s.run()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s.run()
    for t, was in zip((s.tables, s.lens, s.refs, *s.cache), start):
        t.copy_(was)
    for step in range(4):
        parents = [int(p) for p in s.g.integers(0, 6, 6)]
        s.fill(parents)
        before = host_cache(s.cache)
        s.ws.fill_(step)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        s.check(before, parents)


def test_two_streams_at_once(gpu):
    """Two books, caches and workspaces, stepped on two streams with nothing between."""
    import torch
    announce("cache together, two streams")
    steps = [Step(9, 2, 4, 128, 32, 600, 8, "fp16", seed=i) for i in (4, 5)]
    streams = [torch.cuda.Stream() for _ in steps]
    parents, before = [], []
    for s in steps:
        parents.append([int(p) for p in s.g.integers(0, 9, 9)])
        s.fill(parents[-1])
        before.append(host_cache(s.cache))
    torch.cuda.synchronize()
    for s, stream in zip(steps, streams):
        with torch.cuda.stream(stream):
            s.run()
    torch.cuda.synchronize()
    for s, p, b in zip(steps, parents, before):
        s.check(b, p)
