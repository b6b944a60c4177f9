"""Attention over the cache in 64 bits with a bound for every output channel and every logarithm, counted key by
key from the kernels' roundings.

A score: products of D query channels with biased codes of 0 to 255 and the bias's own, each kept exactly and summed in
fp32 in any order: (D + 2) 2^-24 of their magnitudes.  Its logarithm of base 2 with the value scale's added, one
multiply-add: 2^-23 of each with room for the scale's product and the hardware's logarithm.  The exponential: 2^-22.
All of that is a relative error e[j] of a key's share.

A weight goes to fp16 in a unit in which the largest of the row is 2^7 at least (the running maximum never passes
the row's own): half a step is 2^-11 of it, or 2^-25 below 2^-14, which is 2^-32 of the largest.  Products of it with codes
are summed in fp32: 2^-24 of the magnitudes for each step of 32 keys, and for the join and what an instruction rounds
within its own sum 8 more.  Few rows' codes carry a bias of
128, and so does the sum that takes it off again.
"""
import math

import numpy as np


def attention(q, cache, tables, lens, starts, scale, window=0, softcap=0.0, bias=128.0):
    """(out, lse, bound of out, bound of lse); rows that see no key: 0, -infinity, 0, 0."""
    kc, ks, vc, vs = cache
    T, H, D = q.shape
    pages, kv, page = kc.shape[:3]
    out, bound = np.zeros((T, H, D)), np.zeros((T, H, D))
    lse, lse_bound = np.full((T, H), -np.inf), np.zeros((T, H))
    for b in range(len(lens)):
        for row in range(starts[b], starts[b + 1]):
            pos = int(lens[b]) - int(starts[b + 1]) + row
            keys = np.arange(max(0, pos - window + 1) if window else 0, min(pos + 1, tables.shape[1] * page))
            p = tables[b, keys // page]
            keys, p = keys[(p >= 0) & (p < pages)], p[(p >= 0) & (p < pages)]
            if not len(keys):
                continue
            steps = len(keys) / 32.0 + 8.0
            for h in range(H):
                g = h // (H // kv)
                sk, sv = ks[p, g].astype(np.float64), vs[p, g].astype(np.float64)
                k, v = kc[p, g, keys % page].astype(np.float64), vc[p, g, keys % page].astype(np.float64)
                x = q[row, h]
                z = (k @ x) * sk * scale
                off = (D + 2) * 2.0 ** -24 * abs(scale) * sk * ((k + 128) @ np.abs(x) + 128.0 * abs(x.sum()))
                if softcap:
                    z = softcap * np.tanh(z / softcap)
                    off = off + softcap * 2.0 ** -21
                lv = np.abs(np.log2(np.clip(sv, 2.0 ** -80, 2.0 ** 126)))
                off = off + 2.0 ** -23 * (np.abs(z) + 2.0 * lv.max()) + 2.0 ** -22
                m = z.max()
                share = np.exp(z - m)
                total = share.sum()
                share /= total
                e = np.expm1(off)
                e_all = (share * e).sum() + 2.0 ** -24 * steps
                w = share * sv
                out[row, h], lse[row, h] = w @ v, m + math.log(total)
                weight = np.maximum(2.0 ** -11 * w, 2.0 ** -32 * w.max())
                bound[row, h] = ((e + e_all) * w + weight) @ np.abs(v) + 2.0 ** -24 * steps * (w @ (np.abs(v) + 2.0 * bias))
                lse_bound[row, h] = e_all * (1.0 + e_all) + 2.0 ** -22 * (abs(lse[row, h]) + lv.max() + 16.0)
    return out, lse, bound, lse_bound
