"""Plain 64-bit forms of rotary positions, the paged 8-bit cache, its attention
and its book, on numpy arrays and lists: what the GPU results are held against."""
import math

import numpy as np


def frequencies(rotary, base, scaling=None, factor=1.0, original=0.0, low=1.0, high=32.0):
    """(inverse frequencies, magnitude) from their definitions, channel by channel."""
    if scaling == "base":
        base = base * factor ** (rotary / (rotary - 2))
    out = []
    for i in range(rotary // 2):
        f = base ** (-2.0 * i / rotary)
        if scaling == "linear":
            f = f / factor
        elif scaling in ("yarn", "bands"):
            turns = original * f / (2 * math.pi)
            if scaling == "bands":
                keep = (turns - low) / (high - low)
            else:                         # a ramp over i: turns are exponential in it
                keep = math.log(turns / low) / math.log(high / low)
            keep = min(1.0, max(0.0, keep))
            f = keep * f + (1.0 - keep) * f / factor
        out.append(f)
    return np.array(out), 0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0


def rope(x, positions, inv_freq, magnitude=1.0, layout="half", inverse=False):
    """x [T][heads][dim] float64, inv_freq as it is held (fp32)."""
    n = len(inv_freq)
    t = positions.astype(np.float64)[:, None] * inv_freq.astype(np.float64)
    cos, sin = magnitude * np.cos(t)[:, None], magnitude * np.sin(t)[:, None] * (-1.0 if inverse else 1.0)
    out = x.copy()
    a, b = (np.s_[..., :n], np.s_[..., n:2 * n]) if layout == "half" else (np.s_[..., 0:2 * n:2], np.s_[..., 1:2 * n:2])
    out[a], out[b] = x[a] * cos - x[b] * sin, x[b] * cos + x[a] * sin
    return out


def places(starts, lens, tokens):
    """(sequence, position) of each row; sequence -1 behind the last."""
    got = [(-1, 0)] * tokens
    for b in range(len(lens)):
        for j in range(starts[b], starts[b + 1]):
            got[j] = (b, lens[b] - starts[b + 1] + j)
    return got


def append(x, codes, scales, tables, where, page):
    """The blocks that rows x [T][kv][dim] at `where` reach: {(page, head): (exact
    scale, {slot: exact code before rounding})}; codes and scales as they are before."""
    pages = scales.shape[0]
    blocks = {}
    for row, (b, pos) in enumerate(where):
        if b < 0 or pos < 0 or pos // page >= tables.shape[1]:
            continue
        p = tables[b, pos // page]
        if 0 <= p < pages:
            blocks.setdefault(p, {})[pos % page] = row
    out = {}
    for p, rows in blocks.items():
        first = min(rows)
        for h in range(x.shape[1]):
            top = max(np.abs(x[r, h]).max() for r in rows.values()) / 127.0
            was = float(scales[p, h]) if first > 0 else 0.0
            now = max(was, top)
            want = {s: x[r, h] / now if now > 0 else 0.0 * x[r, h] for s, r in rows.items()}
            if now > was:
                want.update({s: codes[p, h, s].astype(np.float64) * (was / now) for s in range(first)})
            out[p, h] = now, want
    return out


def read(codes, scales, tables, where, page):
    out = np.zeros((len(where), codes.shape[1], codes.shape[3]))
    for row, (b, pos) in enumerate(where):
        if b >= 0 and 0 <= pos < tables.shape[1] * page:
            p = tables[b, pos // page]
            if 0 <= p < scales.shape[0]:
                out[row] = codes[p, :, pos % page].astype(np.float64) * scales[p].astype(np.float64)[:, None]
    return out


def attention(q, cache, tables, lens, starts, scale, window=0, softcap=0.0):
    """(out, lse, bound) for q [T][heads][dim] float64.  bound: what the kernels' roundings
    may move `out` by before it is rounded itself.

    Scores: fp32 sums of D products of q with codes of up to 255 (biased), in any order, (D + 2) 2^-24 of the
    sum of magnitudes; one multiply-add, the exponential and the scales' logarithm 2^-20 with room.  Weights
    times the value scale are rounded to fp16: half a step, 2^-11 relative, or 2^-25 of a unit in which the
    largest one is at least 2^-2 (the running maximum is set at most 2^2 above it), 2^-23 of that one; then D-wide sums in fp32."""
    kc, ks, vc, vs = cache
    T, H, D = q.shape
    pages, kv, page = kc.shape[:3]
    out, lse, bound = np.zeros((T, H, D)), np.full((T, H), -np.inf), np.zeros((T, H, D))
    for b in range(len(lens)):
        for row in range(starts[b], starts[b + 1]):
            pos = lens[b] - starts[b + 1] + row
            lo = max(0, pos - window + 1) if window else 0
            keys = [j for j in range(lo, min(pos + 1, tables.shape[1] * page)) if 0 <= tables[b, j // page] < pages]
            if not keys:
                continue
            at, slot = tables[b, np.array(keys) // page], np.array(keys) % page
            for h in range(H):
                g = h // (H // kv)
                sk, sv = ks[at, g].astype(np.float64), vs[at, g].astype(np.float64)
                k, codes = kc[at, g, slot].astype(np.float64) * sk[:, None], vc[at, g, slot].astype(np.float64)
                v = codes * sv[:, None]
                z = k @ q[row, h] * scale
                if softcap:
                    z = softcap * np.tanh(z / softcap)
                m = z.max()
                p = np.exp(z - m)
                total = p.sum()
                p = p / total
                out[row, h], lse[row, h] = p @ v, m + math.log(total)
                score = (D + 2) * 2.0 ** -24 * abs(scale) * np.abs(q[row, h]).sum() * 255.0 * sk.max()
                # capped: cap - 2 cap r, r = 1 / (1 + z) near 1/2 with z rounded by 2^-23, the sum by 2^-24 and the
                # reciprocal by 2^-23, and the cap's sum with a logarithm by 2^-24: cap (2^-24 + 2^-24 + 2^-23 + 2^-24) < cap 2^-21
                score += 2.0 ** -20 * (1.0 + (softcap or 0.0) / 2.0)
                weight = 2.0 ** -11 + 2.0 * math.expm1(score) + 2.0 ** -20 * (2.0 + abs(np.log2(np.maximum(sv, 2.0 ** -100))).max())
                bound[row, h] = weight * (p @ np.abs(v)) + 2.0 ** -23 * (p * sv).max() * np.abs(codes).sum(0)
                bound[row, h] += 2.0 ** -20 * 128.0 * (p @ sv)      # the bias of 128 leaves fp32 sums
    return out, lse, bound


class Book:
    """A cache's book kept in lists."""

    def __init__(self, rows, lens, refs, page):
        self.page, self.lens, self.refs = page, list(lens), list(refs)
        self.rows = [list(r[:self.count(n)]) for r, n in zip(rows, lens)]

    def count(self, n):
        return -(-n // self.page)

    def fork(self, parents):
        B = len(self.rows)
        rows = [list(self.rows[p]) if 0 <= p < B else [] for p in parents]
        lens = [self.lens[p] if 0 <= p < B else 0 for p in parents]
        for r in rows:
            for p in r:
                if 0 <= p < len(self.refs):
                    self.refs[p] += 1
        for r in self.rows:
            for p in r:
                if 0 <= p < len(self.refs):
                    self.refs[p] -= 1
        self.rows, self.lens = rows, lens

    def reserve(self, counts, width):
        """(pairs, status)"""
        B = len(self.rows)
        counts = [max(c, 0) for c in counts]
        pairs = [(-1, -1)] * B
        over = [self.count(n + c) > width for n, c in zip(self.lens, counts)]
        writers = {}
        for b in range(B):
            if not over[b] and counts[b] and self.lens[b] % self.page and self.refs[self.rows[b][-1]] > 1:
                writers.setdefault(self.rows[b][-1], []).append(b)
        copying = set()
        for p, who in writers.items():
            copying.update(who[1:] if len(who) == self.refs[p] else who)
        fresh = [0 if over[b] else self.count(self.lens[b] + counts[b]) - len(self.rows[b]) + (b in copying)
                 for b in range(B)]
        free = [p for p, r in enumerate(self.refs) if r == 0]
        status = [max(0, sum(fresh) - len(free)), sum(over)]
        if any(status):
            return pairs, status
        for b in range(B):
            if b in copying:
                src, dst = self.rows[b][-1], free.pop(0)
                pairs[b], self.rows[b][-1] = (src, dst), dst
                self.refs[src] -= 1
                self.refs[dst] = 1
            self.lens[b] += counts[b]
            while len(self.rows[b]) < self.count(self.lens[b]):
                self.rows[b].append(free.pop(0))
                self.refs[self.rows[b][-1]] = 1
        return pairs, status

    def compact(self):
        """moves"""
        used = [p for p, r in enumerate(self.refs) if r > 0]
        holes = [p for p in range(len(used)) if self.refs[p] <= 0]
        moves = list(zip([p for p in used if p >= len(used)], holes))
        to = dict(moves)
        self.rows = [[to.get(p, p) for p in r] for r in self.rows]
        for src, dst in moves:
            self.refs[dst], self.refs[src] = self.refs[src], 0
        return moves

    def table(self, width):
        return [r + [-1] * (width - len(r)) for r in self.rows]
