"""The attention half of a quantized decoder block over a paged 8-bit cache.

    python examples/cached_attention.py [--steps 6] [--check]

Prompts are read, every prompt is forked into beams that share its pages, and the
beams then decode token by token:

    lens += n              cache_reserve          pages for the new tokens, shared ones replaced
                           cache_copy_pages       ... by copies
    r, q, s                norm_gate_residual     norm + residual, 8-bit codes
    qkv                    gemm_w8a8              the fused q/k/v projection of them
    q                      cache_append           q and k turned by their places, k and v into the cache
    o                      cache_attention        over each row's pages
    block output           linear_w8a8            the output projection

After each step the beams are reordered (cache_fork), and at the end the cache is
compacted (cache_compact, cache_copy_pages).  Weights are random.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import weight_only_quantization_pack_amd as awq  # noqa: E402


class Attention:
    """One layer's attention with its cache.  Rows of a call are the last tokens of the
    table's sequences."""

    def __init__(self, width=512, heads=8, kv=2, dim=64, page=16, pages=256, table=16, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def weights(rows, cols):
            return awq.quantize_rows((cols ** -0.5 * torch.randn(rows, cols, generator=g, device=device)).half())

        self.heads, self.kv, self.dim, self.page = heads, kv, dim, page
        self.norm = (1.0 + 0.1 * torch.randn(width, generator=g, device=device)).half()
        self.qkv, self.out = weights((heads + 2 * kv) * dim, width), weights(width, heads * dim)
        self.inv_freq, self.magnitude = awq.rope_frequencies(dim, 500000.0, scaling="bands", factor=8.0,
                                                             original_length=8192.0, low=1.0, high=4.0, device=device)
        self.cache = awq.empty_cache(pages, kv, page, dim, device=device)
        self.tables = torch.full((1, table), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(1, dtype=torch.int32, device=device)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=device)

    def fork(self, parents):
        """Table row b becomes row parents[b] (-1: empty)."""
        parents = torch.tensor(parents, dtype=torch.int32, device=self.refs.device)
        self.tables, self.lens = awq.cache_fork(self.tables, self.lens, self.refs, parents, self.page)

    def compact(self):
        moves, count = awq.cache_compact(self.tables, self.lens, self.refs, self.page)
        awq.cache_copy_pages(self.cache, moves, count=count)

    def __call__(self, x, residual, new):
        """(residual stream, block output) of fp16 rows [sum(new)][width], new[b] of them for table row b."""
        counts = torch.tensor(new, dtype=torch.int32, device=x.device)
        pairs, short = awq.cache_reserve(self.tables, self.lens, self.refs, counts, self.page)
        if bool(short.any()):
            raise RuntimeError("the cache is full")
        awq.cache_copy_pages(self.cache, pairs)
        starts = torch.zeros(len(new) + 1, dtype=torch.int32, device=x.device)
        starts[1:] = counts.cumsum(0)
        r, q8, scales = awq.norm_gate_residual(x, residual, self.norm, quantize=True)
        qkv = awq.gemm_w8a8(q8, scales, *self.qkv).view(x.shape[0], self.heads + 2 * self.kv, self.dim)
        h = self.heads
        q = awq.cache_append(qkv[:, :h], qkv[:, h:h + self.kv], qkv[:, h + self.kv:], self.cache, self.tables, self.lens,
                             starts, inv_freq=self.inv_freq, magnitude=self.magnitude)
        o = awq.cache_attention(q, self.cache, self.tables, self.lens, starts, max_new=max(new))
        return r, awq.linear_w8a8(o.view(x.shape[0], -1), *self.out)


class Plain:
    """The same with every row's own keys and values in 64 bits, without a cache."""

    def __init__(self, layer):
        self.layer, self.rows = layer, [[]]

    def fork(self, parents):
        self.rows = [list(self.rows[p]) if p >= 0 else [] for p in parents]

    def __call__(self, x, residual, new):
        L, out, at = self.layer, [], 0
        r = residual.double() + x.double()
        n = r / torch.sqrt((r * r).mean(-1, keepdim=True) + 1e-6) * L.norm.double()
        qkv = (n @ (L.qkv[0].double() * L.qkv[1].double()[:, None]).t()).view(len(x), -1, L.dim)
        half = L.dim // 2
        for b, count in enumerate(new):
            for t in range(at, at + count):
                angle = len(self.rows[b]) * L.inv_freq.double()
                turn = qkv[t, :L.heads + L.kv]
                a, c = turn[:, :half], turn[:, half:]
                turned = torch.cat([a * angle.cos() - c * angle.sin(), c * angle.cos() + a * angle.sin()], -1)
                self.rows[b].append((turned[L.heads:], qkv[t, L.heads + L.kv:]))
                k, v = (torch.stack(m).repeat_interleave(L.heads // L.kv, 1) for m in zip(*self.rows[b]))
                p = torch.softmax(torch.einsum("hd,shd->hs", turned[:L.heads], k) * L.dim ** -0.5, -1)
                out.append((p[:, :, None] * v.transpose(0, 1)).sum(1).reshape(-1))
            at += count
        o = torch.stack(out)
        return r, o @ (L.out[0].double() * L.out[1].double()[:, None]).t()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=6, help="tokens that the beams decode")
    ap.add_argument("--check", action="store_true", help="compare with attention in 64 bits on unquantized keys and values")
    a = ap.parse_args(argv)
    layer = Attention()
    plain = Plain(layer)
    g = torch.Generator(device="cuda").manual_seed(1)
    worst = 0.0

    def both(what, *args):
        getattr(layer, what)(*args)
        getattr(plain, what)(*args)

    def step(new):
        nonlocal worst
        x, residual = (torch.randn(sum(new), layer.norm.numel(), generator=g, device="cuda").half() for _ in range(2))
        r, y = layer(x, residual, new)
        if a.check:
            worst = max([worst] + [float((p.double() - w).norm() / w.norm()) for p, w in zip((r, y), plain(x, residual, new))])

    both("fork", [-1, -1])                       # two sequences
    step([37, 20])                               # their prompts
    both("fork", [0, 0, 0, 1, 1, 1])             # three beams each, on shared pages
    for i in range(a.steps):
        step([1] * 6)
        both("fork", [(b + i) % 3 if b < 3 else 3 + (b * i) % 3 for b in range(6)])
    both("fork", [2, -1, -1, 3, 4, -1])          # some are done
    layer.compact()
    step([1, 0, 0, 1, 5, 0])                     # and one reads on
    used = int((layer.refs > 0).sum())
    print(f"{used} pages in use at the front of {layer.refs.numel()}, lengths {layer.lens.tolist()}")
    if a.check:
        print(f"relative difference from 64 bits without quantization: {worst:.2e}")
    return worst


if __name__ == "__main__":
    sys.exit(1 if main() > 5e-2 else 0)
