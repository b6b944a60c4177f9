"""Sequences and caches for the GPU tests of the paged cache."""
import numpy as np

import weight_only_quantization_pack_amd as awq

DTYPES = ["fp16", "bf16"]


def dtype_of(name):
    import torch
    return {"fp16": torch.float16, "bf16": torch.bfloat16}[name]


def gpu(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def ints(values):
    return gpu(np.array(values, dtype=np.int32))


class Case:
    """Sequences of (new, past) tokens over a cache of random codes with scattered
    pages; `bad`: (sequence, page of it, value) entries put into the table."""

    def __init__(self, pairs, heads, kv, dim, page, dtype="fp16", seed=0, spare=2, width=None, bad=(), lens=None):
        g = np.random.default_rng(seed)
        self.heads, self.kv, self.dim, self.page, self.dtype = heads, kv, dim, page, dtype_of(dtype)
        self.new = [n for n, _ in pairs]
        self.lens = np.array([n + p for n, p in pairs] if lens is None else lens, dtype=np.int32)
        self.starts = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.T = int(self.starts[-1])
        need = [-(-(n + p) // page) for n, p in pairs]
        self.pages = sum(need) + spare
        ids = g.permutation(self.pages)
        W = width or max(need + [1])
        self.tables = np.full((len(pairs), W), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.tables[b, :n] = ids[at:at + n]
            at += n
        for b, w, value in bad:
            self.tables[b, w] = value
        shape = (self.pages, kv, page, dim)
        self.cache = [c for _ in range(2) for c in (
            np.clip(np.rint(32 * g.standard_normal(shape)), -127, 127).astype(np.int8),
            (0.03 * np.exp(0.5 * g.standard_normal(shape[:2]))).astype(np.float32))]
        self.g = g

    def rows(self, heads, spread=1.0, tokens=None):
        """[T][heads][dim] on the GPU in the case's type, channels of different sizes."""
        x = spread * self.g.standard_normal((self.T if tokens is None else tokens, heads, self.dim))
        return gpu((x * np.exp(0.5 * self.g.standard_normal((heads, self.dim)))).astype(np.float32)).to(self.dtype)

    def on_gpu(self):
        """(cache, tables, lens, starts)"""
        return tuple(gpu(c) for c in self.cache), gpu(self.tables), gpu(self.lens), gpu(self.starts)


def host_cache(cache):
    return [c.cpu().numpy() for c in cache]


def freq(rotary, base=10000.0, **scaling):
    return awq.rope_frequencies(rotary, base, **scaling)
