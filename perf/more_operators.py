"""Cases of the operators around a key and value cache held in 8 bits: what a decoder block needs between
its 8-bit projections (perf/operators.py).

The cache is paged.  A page holds `page` consecutive tokens of one sequence for every kv head as int8 codes
[kv][page][dim], keys and values apart, each with one fp32 scale for its block of tokens and head: a value is
code * scale.  Row b of `tables` lists the pages of sequence b in order and `lens[b]` counts its tokens.

Four operators, each with its cases, its inputs, its plain form and its 64-bit definition:

  rope    rotary positions of the rows of a projection: for every pair (a, b) of the first `rotary` channels
          of a head and the angle t = position * inv_freq[i]
              a' = m (a cos t - b sin t),   b' = m (b cos t + a sin t)
          pairs are (i, i + rotary / 2) ("half") or (2i, 2i + 1) ("interleaved"); m is the magnitude that
          long-context scaling asks for
  append  rope of q and k, and k and v into the cache.  The block of a page that new tokens x reach gets the scale
              s' = max(s, max|x| / 127)          (s = 0 for a block that held no tokens)
          its older codes become rint(code * s / s'), the new ones rint(x / s').  What is written is then
          read back as the values that it stands for
  attend  attention of each sequence's last n tokens over its cached keys and values (causal; within a
          window; with capped scores):
              o = sum_j p_j v_j,  p = softmax_j(cap * tanh(scale * q.k_j / cap))
  pages   the bookkeeping of a cache whose pages sequences share: rows are forked, reordered and dropped
          by parent indices (beams), rows grow by some tokens (the lowest free pages are taken; a shared page
          that is written to is copied first), and scattered pages are moved to the front ("compact")

`run` takes what `prepare` gives through the plain form (elementary torch operations in 32 bits, angles in
64, rounded once) where `own` is false, and through the library's entry points where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the queries of one token of a 4096-wide decoder: launch latency is the whole cost
        dict(name="rope_one_token", op="rope", tokens=1, heads=32, dim=128, rotary=128, layout="half",
             dtype="fp16", far=4096, scaling="none"),
        # an odd prompt chunk far out in a long context, half of each head rotated in adjacent pairs
        dict(name="rope_chunk_partial", op="rope", tokens=4099, heads=64, dim=128, rotary=64,
             layout="interleaved", dtype="bf16", far=1000000, scaling="yarn"),
        # a decode batch: one token of each sequence into a partly filled page
        dict(name="append_decode", op="append", seqs=64, new_lo=1, new_hi=1, past_lo=16, past_hi=4000,
             heads=32, kv=8, dim=128, page=64, rotary=128, layout="half", dtype="fp16", scaling="none"),
        # three ragged prompt chunks behind what their sequences hold already
        dict(name="append_chunks", op="append", seqs=3, new_lo=333, new_hi=2047, past_lo=100, past_hi=8000,
             heads=32, kv=8, dim=128, page=16, rotary=128, layout="half", dtype="bf16", scaling="llama3"),
        # a long prompt of a wide model
        dict(name="append_prompt", op="append", seqs=1, new_lo=16384, new_hi=16384, past_lo=0, past_hi=0,
             heads=64, kv=8, dim=128, page=64, rotary=128, layout="half", dtype="bf16", scaling="none"),
        # one token over a short context: latency
        dict(name="attend_one_token", op="attend", seqs=1, new_lo=1, new_hi=1, past_lo=130, past_hi=130,
             heads=32, kv=8, dim=128, page=64, window=0, cap=0.0, dtype="fp16"),
        # a decode batch of a wide model over contexts of different lengths: the cache's read is the cost
        dict(name="attend_batch", op="attend", seqs=64, new_lo=1, new_hi=1, past_lo=200, past_hi=8000,
             heads=64, kv=8, dim=128, page=64, window=0, cap=0.0, dtype="bf16"),
        # one token over a long context: the read has to be spread over the card
        dict(name="attend_long", op="attend", seqs=1, new_lo=1, new_hi=1, past_lo=131071, past_hi=131071,
             heads=32, kv=8, dim=128, page=64, window=0, cap=0.0, dtype="fp16"),
        # prompt chunks with a past, small pages, a sliding window and capped scores
        dict(name="attend_chunks", op="attend", seqs=3, new_lo=260, new_hi=1100, past_lo=500, past_hi=6000,
             heads=32, kv=8, dim=128, page=16, window=4096, cap=50.0, dtype="bf16"),
        # a long prompt: the matrix pipes are the cost
        dict(name="attend_prompt", op="attend", seqs=1, new_lo=8192, new_hi=8192, past_lo=0, past_hi=0,
             heads=32, kv=8, dim=128, page=64, window=0, cap=0.0, dtype="bf16"),
        # one step of a beam search: rows reordered, one token more, shared pages copied before they are written
        dict(name="pages_beams", op="pages", kind="beams", groups=16, beams=4, past_lo=100, past_hi=2000,
             new=1, kv=8, dim=128, page=64, layers=4, spare=256),
        # a fragmented cache moved to the front: copies of whole pages in every layer
        dict(name="pages_compact", op="pages", kind="compact", groups=96, beams=1, past_lo=500, past_hi=4000,
             new=0, kv=8, dim=128, page=64, layers=8, spare=2000),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in lo..hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return min(hi, max(lo, int(v) // step * step))


def _lengths(n, lo, hi):
    """n lengths spread over the logarithm of lo..hi, the same for every seed (their order is not)."""
    return [int(lo * (hi / lo) ** ((i + 1) * 0.6180339887 % 1.0) + 0.5) if lo > 0 else (hi * (i + 1) // n)
            for i in range(n)]


def _pairs(c):
    """(new, past) tokens of each sequence."""
    return list(zip(_lengths(c["seqs"], c["new_lo"], c["new_hi"]), _lengths(c["seqs"], c["past_lo"], c["past_hi"])[::-1]))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "attend", "attend", "attend", "pages"])
    dtype = rng.choice(["fp16", "bf16"])
    dim = rng.choice([64, 96, 128, 128, 192, 256])
    rotary = rng.choice([dim, dim, dim // 2 // 16 * 16])
    layout, scaling = rng.choice(["half", "interleaved"]), rng.choice(["none", "linear", "yarn", "llama3"])
    if op == "rope":
        heads = _log(rng, 1, 64)
        return dict(op=op, tokens=_log(rng, 1, max(1, min(16384, 4099 * 64 * 128 // (heads * dim)))), heads=heads,
                    dim=dim, rotary=rotary, layout=layout, dtype=dtype, far=_log(rng, 100, 1000000), scaling=scaling)
    kv, group = rng.choice([1, 2, 3, 4, 8, 8]), rng.choice([1, 2, 4, 4, 5, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        seqs = _log(rng, 1, 256)
        most = max(1, 16384 * 80 * 128 // (seqs * (group + 2) * kv * dim))
        hi = rng.choice([1, _log(rng, 1, min(most, 16384))])
        past = _log(rng, 1, max(1, 131072 // seqs))
        return dict(op=op, seqs=seqs, new_lo=max(1, hi // rng.randint(1, 6)), new_hi=hi, past_lo=past // rng.randint(1, 30),
                    past_hi=past, heads=kv * group, kv=kv, dim=dim, page=page, rotary=rotary, layout=layout,
                    dtype=dtype, scaling=scaling)
    if op == "attend":
        kind = rng.choice(["decode", "decode", "verify", "chunk"])
        seqs = _log(rng, 1, 256 if kind != "chunk" else 8)
        hi = 1 if kind == "decode" else rng.randint(2, 8) if kind == "verify" else _log(rng, 16, 4096)
        # the cache (gathered in 32 bits by the plain form) and the plain form's scores stay within the listed ones'
        past = _log(rng, 1, max(1, min(131072, 500000 * 1024 // (seqs * kv * dim))))
        while hi > 1 and 8 * seqs * kv * group * hi * (hi + past) > 32 * 8192 ** 2:
            hi, past = max(1, hi // 2), max(1, past // 2)
        return dict(op=op, seqs=seqs, new_lo=max(1, hi // rng.randint(1, 4)), new_hi=hi,
                    past_lo=max(1, past // rng.randint(1, 30)), past_hi=past, heads=kv * group, kv=kv, dim=dim, page=page,
                    window=rng.choice([0, 0, _log(rng, 16, 8192)]), cap=rng.choice([0.0, 0.0, 30.0]), dtype=dtype)
    kind = rng.choice(["beams", "compact"])
    groups = _log(rng, 1, 64)
    past = _log(rng, 20, max(20, 96 * 2000 // groups))
    return dict(op=op, kind=kind, groups=groups, beams=rng.randint(2, 8) if kind == "beams" else 1,
                past_lo=max(1, past // 10), past_hi=past, new=rng.choice([1, 1, 5, 70]) if kind == "beams" else 0,
                kv=kv, dim=dim, page=rng.choice([32, 64, 128]), layers=rng.choice([1, 2, 4]), spare=_log(rng, 64, 1024))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _frequencies(rotary, scaling):
    """(inverse frequencies fp32, magnitude) of a base of 10000 (500000 scaled), stretched for long contexts."""
    n = rotary // 2
    base = 10000.0 if scaling == "none" else 500000.0
    f = [base ** (-i / n) for i in range(n)]
    if scaling == "linear":
        f = [v / 4.0 for v in f]
    elif scaling == "llama3":        # long wavelengths by 8, short ones not, between them by degrees
        part = [min(1.0, max(0.0, (8192 * v / (2 * math.pi) - 1.0) / 3.0)) for v in f]
        f = [v / 8.0 * (1.0 - p) + v * p for v, p in zip(f, part)]
    elif scaling == "yarn":          # channels that turn over 32 times in 4096 tokens stay, under once are stretched by 16
        lo, hi = (n * math.log(4096 / (t * 2 * math.pi)) / math.log(base) for t in (32.0, 1.0))
        part = [min(1.0, max(0.0, (i - lo) / (hi - lo))) for i in range(n)]
        f = [v / 16.0 * p + v * (1.0 - p) for v, p in zip(f, part)]
    magnitude = 0.1 * math.log(16.0) + 1.0 if scaling == "yarn" else 1.0
    return torch.tensor(f, dtype=torch.float64).to(torch.float32).to(DEV), magnitude


def _heads(g, tokens, heads, dim, dtype):
    """Projected rows whose channels differ in size, as keys' do."""
    return (_randn(g, tokens, heads, dim) * torch.exp(0.5 * _randn(g, heads, dim))).to(dtype)


def _codes(g, *shape):
    """Codes of blocks whose largest value is some four times their spread."""
    return torch.empty(shape, dtype=torch.float16, device=DEV).normal_(0.0, 30.0, generator=g).round_() \
        .clamp_(-127, 127).to(torch.int8)


def _scales(g, *shape):
    return 0.03 * torch.exp(0.3 * _randn(g, *shape))


def _cache(g, pages, c, layers=None):
    """(key codes, key scales, value codes, value scales) of a cache in use."""
    lead = (pages,) if layers is None else (layers, pages)
    return [t for _ in range(2) for t in (_codes(g, *lead, c["kv"], c["page"], c["dim"]), _scales(g, *lead, c["kv"]))]


def _shuffled(g, values):
    order = torch.randperm(len(values), generator=g, device=DEV).tolist()
    return [values[i] for i in order]


def _tables(g, lens, page, spare=0):
    """(tables int32 [B][W], pages): the sequences' pages scattered over the cache, -1 behind a row's last."""
    need = [-(-n // page) for n in lens]
    pages = max(1, sum(need) + spare)
    ids = torch.randperm(pages, generator=g, device=DEV).tolist()
    rows, at = [], 0
    for n in need:
        rows.append(ids[at:at + n] + [-1] * (max(need) - n))
        at += n
    return _ints(rows), pages


def _ragged(g, c):
    """Sequences with their new tokens: lens counts them, starts has the new ones' offsets."""
    pairs = _shuffled(g, _pairs(c))
    new = [n for n, _ in pairs]
    lens = [n + p for n, p in pairs]
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    tables, pages = _tables(g, lens, c["page"], spare=3)
    return dict(lens=_ints(lens), starts=_ints(starts), tables=tables, tokens=starts[-1], most_new=max(new),
                most_len=max(lens), cache=_cache(g, pages, c)), new, lens


def _book(c, tables, lens, refs):
    """One tensor that holds a cache's book, so that one copy keeps it: [tables | lens | refs]."""
    flat = [v for row in tables for v in row] + lens + refs
    return _ints(flat), (len(tables), len(tables[0]), len(refs))


def _beams(g, c):
    """Groups of beams that share their prompt's pages and have tails of their own; rows to come from them."""
    page, tables, lens, want = c["page"], [], [], []
    rows = c["groups"] * c["beams"]
    past = _shuffled(g, _lengths(c["groups"], c["past_lo"], c["past_hi"]))
    width = -(-(max(past) + c["new"]) // page)
    need = sum((n // 2 // page) + c["beams"] * (-(-n // page) - n // 2 // page) for n in past)
    pages = need + rows * (2 + c["new"] // page) + c["spare"]
    ids, at = torch.randperm(pages, generator=g, device=DEV).tolist(), 0
    refs = [0] * pages
    for n in past:
        shared, count = n // 2 // page, -(-n // page)
        prompt = ids[at:at + shared]
        at += shared
        for _ in range(c["beams"]):
            tail = ids[at:at + count - shared]
            at += count - shared
            tables.append(prompt + tail + [-1] * (width - count))
            lens.append(n)
            for p in prompt + tail:
                refs[p] += 1
    pick = torch.randint(0, c["beams"], (rows,), generator=g, device=DEV).tolist()
    done = set(torch.randperm(c["groups"], generator=g, device=DEV).tolist()[:c["groups"] // 8])
    for b in range(rows):
        group = b // c["beams"]
        want.append(-1 if group in done else group * c["beams"] + pick[b])
    return tables, lens, refs, want, pages


def _scattered(g, c):
    """Sequences whose pages lie anywhere in a cache that is partly free."""
    lens = _shuffled(g, _lengths(c["groups"], c["past_lo"], c["past_hi"]))
    tables, pages = _tables(g, lens, c["page"], spare=c["spare"])
    tables = tables.tolist()
    refs = [0] * pages
    for row in tables:
        for p in row:
            if p >= 0:
                refs[p] += 1
    return tables, lens, refs, pages


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case=dict(c))
    if c["op"] == "rope":
        s["x"] = _heads(g, c["tokens"], c["heads"], c["dim"], DTYPES[c["dtype"]])
        first = int(torch.randint(max(1, c["far"] // 2), c["far"] + 1, (1,), generator=g, device=DEV))
        s["positions"] = torch.arange(first, first + c["tokens"], device=DEV, dtype=torch.int32)
        s["inv_freq"], s["magnitude"] = _frequencies(c["rotary"], c["scaling"])
    elif c["op"] == "append":
        dtype = DTYPES[c["dtype"]]
        ragged, new, lens = _ragged(g, c)
        s.update(ragged)
        # one projection's rows [q | k | v], as a fused layer leaves them
        s["qkv"] = _heads(g, s["tokens"], c["heads"] + 2 * c["kv"], c["dim"], dtype)
        s["inv_freq"], s["magnitude"] = _frequencies(c["rotary"], c["scaling"])
        back = [0]                    # every token of the pages that the new ones reach
        for n, total in zip(new, lens):
            back.append(back[-1] + n + (total - n) % c["page"])
        s["read_starts"], s["read_tokens"] = _ints(back), back[-1]
    elif c["op"] == "attend":
        ragged, _, _ = _ragged(g, c)
        s.update(ragged)
        s["q"] = (2.5 * _randn(g, s["tokens"], c["heads"], c["dim"])).to(DTYPES[c["dtype"]])
        s["scale"] = c["dim"] ** -0.5
    elif c["kind"] == "beams":
        tables, lens, refs, parents, pages = _beams(g, c)
        s["book"], s["sizes"] = _book(c, tables, lens, refs)
        s["parents"] = _ints(parents)
        s["new"] = _ints([c["new"] if p >= 0 else 0 for p in parents])
        s["cache"] = _cache(g, pages, c, c["layers"])
    else:
        tables, lens, refs, pages = _scattered(g, c)
        s["book"], s["sizes"] = _book(c, tables, lens, refs)
        s["cache"] = _cache(g, pages, c, c["layers"])
    return s


def _open(s):
    """(tables, lens, refs) of a copy of the book: the step before stays, to go back to."""
    rows, width, pages = s["sizes"]
    tables, lens, refs = s["book"].clone().split([rows * width, rows, pages])
    return tables.view(rows, width), lens, refs


# ---------------------------------------------------------------------------
# plain forms: 32 bits (angles in 64), one rounding at the end
# ---------------------------------------------------------------------------
def _plain_rotate(x, positions, inv_freq, magnitude, layout):
    """The rows x [T][heads][dim] rotated, in 32 bits."""
    x = x.float()
    angle = positions.double()[:, None] * inv_freq.double()
    cos, sin = ((magnitude * f(angle)).float()[:, None, :] for f in (torch.cos, torch.sin))
    n = 2 * inv_freq.numel()
    if layout == "half":
        a, b = x[..., :n // 2], x[..., n // 2:n]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., n:]], dim=-1)
    a, b = x[..., 0:n:2], x[..., 1:n:2]
    turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([turned, x[..., n:]], dim=-1)


def _plain_places(starts, lens, tokens):
    """(sequence, position) of each of the `tokens` last tokens of the sequences."""
    t = torch.arange(tokens, device=DEV)
    seq = torch.searchsorted(starts[1:].long(), t, right=True)
    return seq, lens[seq].long() - starts[seq + 1].long() + t


def _plain_write(codes, scales, x, seq, pos, s, page):
    """x [T][kv][dim] in 32 bits into the blocks of its positions."""
    tables, lens, starts = s["tables"], s["lens"].long(), s["starts"].long()
    pages, kv = scales.shape
    at = tables[seq, pos // page].long()
    top = torch.zeros(pages, kv, device=DEV).scatter_reduce_(0, at[:, None].expand(-1, kv), x.abs().amax(dim=-1), "amax")
    first = lens - (starts[1:] - starts[:-1])
    held = (first % page != 0) & (first < lens)
    old = tables[held, first[held] // page].long()
    before = torch.zeros_like(scales)
    before[old] = scales[old]
    after = torch.maximum(before, top / 127.0)
    kept = torch.arange(page, device=DEV)[None, :] < (first[held] % page)[:, None]
    shrink = (before[old] / torch.where(after[old] > 0, after[old], torch.ones_like(after[old])))[:, :, None, None]
    was = codes[old].float()
    codes[old] = torch.where(kept[:, None, :, None], torch.round(was * shrink), was).to(torch.int8)
    scales[at] = after[at]
    step = after[at][:, :, None]
    q = torch.where(step > 0, torch.round(x / torch.where(step > 0, step, torch.ones_like(step))), torch.zeros_like(x))
    codes[at, :, pos % page, :] = q.clamp(-127, 127).to(torch.int8)


def _plain_append(s, c):
    dtype, h, kv = DTYPES[c["dtype"]], c["heads"], c["kv"]
    seq, pos = _plain_places(s["starts"], s["lens"], s["tokens"])
    turned = _plain_rotate(s["qkv"][:, :h + kv], pos, s["inv_freq"], s["magnitude"], c["layout"])
    kc, ks, vc, vs = s["cache"]
    _plain_write(kc, ks, turned[:, h:], seq, pos, s, c["page"])
    _plain_write(vc, vs, s["qkv"][:, h + kv:].float(), seq, pos, s, c["page"])
    seq, pos = _plain_places(s["read_starts"], s["lens"], s["read_tokens"])
    at, slot = s["tables"][seq, pos // c["page"]].long(), pos % c["page"]
    k, v = (codes[at, :, slot].float() * scales[at][:, :, None] for codes, scales in ((kc, ks), (vc, vs)))
    return turned[:, :h].to(dtype), k.to(dtype), v.to(dtype)


def _plain_attend(s, c):
    kc, ks, vc, vs = s["cache"]
    b, h, kv, d = c["seqs"], c["heads"], c["kv"], c["dim"]
    n, span = s["most_new"], s["tables"].shape[1] * c["page"]
    starts, lens = s["starts"].long(), s["lens"].long()
    new = starts[1:] - starts[:-1]
    pages = s["tables"].clamp(min=0).long()
    k, v = ((codes[pages].float() * scales[pages][..., None, None]).permute(0, 2, 1, 3, 4).reshape(b, kv, span, d)
            for codes, scales in ((kc, ks), (vc, vs)))
    j = torch.arange(n, device=DEV)
    row = (starts[:-1, None] + j).clamp(max=s["tokens"] - 1)                 # [b][n], padded with some other row
    q = s["q"].float()[row].view(b, n, kv, h // kv, d).permute(0, 2, 3, 1, 4).reshape(b, kv, h // kv * n, d)
    z = (q @ k.transpose(-1, -2)) * s["scale"]
    if c["cap"]:
        z = torch.tanh(z / c["cap"]) * c["cap"]
    at = torch.arange(span, device=DEV)
    place = (lens - new)[:, None] + j                                        # [b][n]
    seen = (at <= place[:, :, None]) & (j[:, None] < new[:, None, None])
    if c["window"]:
        seen = seen & (at > place[:, :, None] - c["window"])
    z = z.view(b, kv, h // kv, n, span).masked_fill_(~seen[:, None, None], -math.inf)
    top = z.amax(dim=-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = z.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    o = (p.view(b, kv, -1, span) @ v).view(b, kv, h // kv, n, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    seq, pos = _plain_places(s["starts"], s["lens"], s["tokens"])
    return o.permute(0, 3, 1, 2, 4).reshape(b, n, h, d)[seq, pos - (lens - new)[seq]].to(DTYPES[c["dtype"]])


def _plain_refs(refs, table, valid, sign):
    return refs.index_add_(0, table[valid].long(), torch.full_like(table[valid], sign))


def _plain_beams(s, c):
    page = c["page"]
    tables, lens, refs = _open(s)
    width, pages, rows = tables.shape[1], refs.shape[0], tables.shape[0]
    cell = torch.arange(width, device=DEV)
    # rows from their parents
    parents = s["parents"].long()
    alive = parents >= 0
    grown = torch.where(alive[:, None], tables[parents.clamp(min=0)], torch.full_like(tables, -1))
    length = torch.where(alive, lens[parents.clamp(min=0)], torch.zeros_like(lens))
    refs = _plain_refs(refs, grown, cell < (-(-length // page))[:, None], 1)
    refs = _plain_refs(refs, tables, cell < (-(-lens // page))[:, None], -1)
    # room for new tokens: whole pages, and a copy of a last page that others hold too; the first of a page's
    # writers keeps it where no one else holds it
    new = s["new"]
    have, want = -(-length // page), -(-(length + new) // page)
    last = grown.gather(1, (have - 1).clamp(min=0).long()[:, None])[:, 0].long()
    writes = (new > 0) & (length % page != 0) & (refs[last.clamp(min=0)] > 1)
    same = (last[:, None] == last[None, :]) & writes[:, None] & writes[None, :]
    order = torch.arange(rows, device=DEV)
    first = ~(same & (order[None, :] < order[:, None])).any(dim=1)
    keeps = first & (same.sum(dim=1) == refs[last.clamp(min=0)])
    copies = (writes & ~keeps).int()
    fresh = want - have + copies
    offset = fresh.cumsum(0) - fresh
    free = torch.sort((refs != 0).int(), stable=True).indices.int()
    fits = (fresh.sum() <= (refs == 0).sum()) & (want <= width).all()
    short = torch.stack([(fresh.sum() - (refs == 0).sum()).clamp(min=0), (want > width).sum()]).int()
    from_ = (have - copies)[:, None]
    takes = (cell >= from_) & (cell < want[:, None]) & fits
    index = (offset[:, None] + cell - from_).clamp(0, pages - 1).long()
    out = torch.where(takes, free[index], grown)
    copied = (copies > 0) & fits
    pair = torch.where(copied[:, None], torch.stack([last.int(), free[offset.clamp(0, pages - 1).long()]], dim=1),
                       torch.full((rows, 2), -1, dtype=torch.int32, device=DEV))
    refs = _plain_refs(refs, out, takes, 1)
    refs = _plain_refs(refs, last.int(), copied, -1)
    length = torch.where(fits, length + new, length)
    _plain_copy(s["cache"], pair[copied])
    return [out, length, refs, pair, short, *s["cache"]]


def _plain_copy(cache, pairs):
    src, dst = pairs.long().unbind(1)
    for t in cache:
        t[:, dst] = t[:, src]


def _plain_compact(s, c):
    tables, lens, refs = _open(s)
    pages = refs.shape[0]
    used = refs > 0
    count = used.sum()
    at = torch.arange(pages, device=DEV)
    holes, movers = ~used & (at < count), used & (at >= count)
    moves = torch.full((pages, 2), -1, dtype=torch.int32, device=DEV)
    src, dst = at[movers], at[holes]
    moves[:src.shape[0]] = torch.stack([src, dst], dim=1).int()
    to = at.int()
    to[src] = dst.int()
    cell = torch.arange(tables.shape[1], device=DEV) < (-(-lens // c["page"]))[:, None]
    tables = torch.where(cell, to[tables.clamp(min=0).long()], tables)
    refs[dst] = refs[src]
    refs[src] = 0
    _plain_copy(s["cache"], moves[:src.shape[0]])
    return [tables, refs, moves, movers.sum().int()[None], *s["cache"]]


def _plain(s, c):
    if c["op"] == "rope":
        return _plain_rotate(s["x"], s["positions"], s["inv_freq"], s["magnitude"], c["layout"]).to(s["x"].dtype)
    if c["op"] == "append":
        return _plain_append(s, c)
    if c["op"] == "attend":
        return _plain_attend(s, c)
    return _plain_beams(s, c) if c["kind"] == "beams" else _plain_compact(s, c)


# ---------------------------------------------------------------------------
# the library's operators
# ---------------------------------------------------------------------------
def _own(s, c):
    import weight_only_quantization_pack_amd as awq

    if c["op"] == "rope":
        return awq.rope(s["x"], s["positions"], s["inv_freq"], layout=c["layout"], magnitude=s["magnitude"])
    if c["op"] == "append":
        h, kv = c["heads"], c["kv"]
        q, k, v = s["qkv"][:, :h], s["qkv"][:, h:h + kv], s["qkv"][:, h + kv:]
        turned = awq.cache_append(q, k, v, s["cache"], s["tables"], s["lens"], s["starts"], inv_freq=s["inv_freq"],
                                  layout=c["layout"], magnitude=s["magnitude"])
        k, v = awq.cache_read(s["cache"], s["tables"], s["lens"], s["read_starts"], tokens=s["read_tokens"],
                              dtype=DTYPES[c["dtype"]])
        return turned, k, v
    if c["op"] == "attend":
        return awq.cache_attention(s["q"], s["cache"], s["tables"], s["lens"], s["starts"], scale=s["scale"],
                                   window=c["window"], softcap=c["cap"], max_new=s["most_new"], max_len=s["most_len"])
    tables, lens, refs = _open(s)
    if c["kind"] == "beams":
        tables, lens = awq.cache_fork(tables, lens, refs, s["parents"], page_size=c["page"])
        pairs, short = awq.cache_reserve(tables, lens, refs, s["new"], page_size=c["page"])
        awq.cache_copy_pages(s["cache"], pairs, layers=c["layers"])
        return [tables, lens, refs, pairs, short, *s["cache"]]
    moves, count = awq.cache_compact(tables, lens, refs, page_size=c["page"])
    awq.cache_copy_pages(s["cache"], moves, count=count, layers=c["layers"])
    return [tables, refs, moves, count, *s["cache"]]


def run(state):
    return _own(state, state["case"]) if own else _plain(state, state["case"])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "rope":
        n = c["tokens"] * c["heads"] * c["dim"]
        return {"bytes": 4 * n + 4 * c["tokens"], "flops": 6 * c["tokens"] * c["heads"] * c["rotary"] // 2}
    if c["op"] in ("append", "attend"):
        pairs, kv, h, d, page = _pairs(c), c["kv"], c["heads"], c["dim"], c["page"]
    if c["op"] == "append":
        tokens = sum(n for n, _ in pairs)
        old = sum(p % page for _, p in pairs)
        # rows in and queries out, codes out, and read back: codes in and rows out
        back = (tokens + old) * kv * d
        return {"bytes": tokens * d * (4 * h + 4 * kv) + 2 * tokens * kv * d + 2 * back + 4 * back,
                "flops": 3 * tokens * (h + kv) * c["rotary"] + 4 * tokens * kv * d}
    if c["op"] == "attend":
        window = c["window"] or 1 << 60
        keys = scores = 0
        for n, p in pairs:
            keys += min(n + p, n - 1 + window)
            m = min(n, max(0, window - p))                       # rows that see everything before them
            scores += m * p + m * (m + 1) // 2 + (n - m) * window
        tokens = sum(n for n, _ in pairs)
        return {"bytes": 2 * keys * kv * d + 4 * tokens * h * d, "flops": 4 * scores * h * d}
    page_bytes = 2 * c["kv"] * (c["page"] * c["dim"] + 4) * c["layers"]
    lengths = _lengths(c["groups"], c["past_lo"], c["past_hi"])
    if c["kind"] == "beams":
        rows = c["groups"] * c["beams"]
        # a last page is copied by all rows but the first of each surviving beam: on average by those beyond
        # the beams that have a child
        b = c["beams"]
        copies = (c["groups"] - c["groups"] // 8) * (b - b * (1.0 - (1.0 - 1.0 / b) ** b))
        width = -(-(max(lengths) + c["new"]) // c["page"])
        return {"bytes": 2 * copies * page_bytes + 4 * (2 * rows * width + 4 * rows), "flops": 0}
    used = sum(-(-n // c["page"]) for n in lengths)
    pages = used + c["spare"]
    return {"bytes": 2 * used * (1.0 - used / pages) * page_bytes + 16 * pages + 8 * used, "flops": 0}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_rotate(x, positions, inv_freq, magnitude, layout):
    out = x.double().clone()
    n = inv_freq.numel()
    for i in range(n):
        a, b = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
        t = positions.double() * inv_freq[i].double()
        cos, sin = magnitude * torch.cos(t)[:, None], magnitude * torch.sin(t)[:, None]
        u, v = x[..., a].double(), x[..., b].double()
        out[..., a], out[..., b] = u * cos - v * sin, v * cos + u * sin
    return out


def _exact_append(s, c):
    h, kv, page = c["heads"], c["kv"], c["page"]
    lens, starts, back = s["lens"].tolist(), s["starts"].tolist(), s["read_starts"].tolist()
    tables = s["tables"].tolist()
    pos = torch.cat([torch.arange(lens[b] - (starts[b + 1] - starts[b]), lens[b], device=DEV) for b in range(c["seqs"])])
    q, k = (_exact_rotate(x, pos, s["inv_freq"], s["magnitude"], c["layout"])
            for x in (s["qkv"][:, :h], s["qkv"][:, h:h + kv]))
    outs = []
    for x, codes, scales in ((k, *s["cache"][:2]), (s["qkv"][:, h + kv:].double(), *s["cache"][2:])):
        got = torch.empty(s["read_tokens"], kv, c["dim"], dtype=torch.float64, device=DEV)
        for b in range(c["seqs"]):
            n, at = starts[b + 1] - starts[b], back[b]
            first = lens[b] - n
            for w in range(first // page, -(-lens[b] // page)):
                lo, hi = max(first, w * page), min(lens[b], (w + 1) * page)
                held = lo - w * page                             # tokens of the page that were there
                rows = x[starts[b] + lo - first:starts[b] + hi - first].transpose(0, 1)     # [kv][tokens][dim]
                top = rows.abs().amax(dim=(1, 2)) / 127.0
                was = scales[tables[b][w]].double() if held else torch.zeros_like(top)
                now = torch.maximum(was, top)
                safe = torch.where(now > 0, now, torch.ones_like(now))[:, None, None]
                older = torch.round(codes[tables[b][w], :, :held].double() * was[:, None, None] / safe)
                newer = torch.round(rows / safe)
                block = torch.cat([older, newer], dim=1) * now[:, None, None]
                got[at:at + block.shape[1]] = block.transpose(0, 1)
                at += block.shape[1]
        outs.append(got)
    return q, outs[0], outs[1]


def _exact_attend(s, c):
    h, kv, d, page = c["heads"], c["kv"], c["dim"], c["page"]
    lens, starts = s["lens"].tolist(), s["starts"].tolist()
    out = torch.zeros(s["tokens"], h, d, dtype=torch.float64, device=DEV)
    for b in range(c["seqs"]):
        n, total = starts[b + 1] - starts[b], lens[b]
        ids = s["tables"][b, :-(-total // page)].long()
        place = torch.arange(total - n, total, device=DEV)[:, None]
        at = torch.arange(total, device=DEV)[None, :]
        hidden = at > place
        if c["window"]:
            hidden = hidden | (at <= place - c["window"])
        for head in range(kv):
            k, v = ((codes[ids, head].double() * scales[ids, head].double()[:, None, None]).reshape(-1, d)[:total]
                    for codes, scales in (s["cache"][:2], s["cache"][2:]))
            for i in range(head * (h // kv), (head + 1) * (h // kv)):
                z = s["q"][starts[b]:starts[b + 1], i].double() @ k.t() * s["scale"]
                if c["cap"]:
                    z = c["cap"] * torch.tanh(z / c["cap"])
                out[starts[b]:starts[b + 1], i] = torch.softmax(z.masked_fill(hidden, -math.inf), dim=-1) @ v
    return out


def _exact_pages(s, c):
    """The book kept page by page in lists; the cache's pages as they are after the copies."""
    rows, width, pages = s["sizes"]
    flat, page = s["book"].tolist(), c["page"]
    tables = [flat[i * width:(i + 1) * width] for i in range(rows)]
    lens, refs = flat[rows * width:rows * width + rows], flat[rows * width + rows:]
    count = lambda n: -(-n // page)  # noqa: E731
    cache = [t.clone() for t in s["cache"]]
    if c["kind"] == "compact":
        used = [p for p in range(pages) if refs[p]]
        holes = [p for p in range(len(used)) if not refs[p]]
        moves = list(zip([p for p in used if p >= len(used)], holes))
        to = dict(moves)
        for b in range(rows):
            for w in range(count(lens[b])):
                tables[b][w] = to.get(tables[b][w], tables[b][w])
        for src, dst in moves:
            refs[dst], refs[src] = refs[src], 0
            for t in cache:
                t[:, dst] = t[:, src]
        listing = [list(m) for m in moves] + [[-1, -1]] * (pages - len(moves))
        return [_ints(tables), _ints(refs), _ints(listing), _ints([len(moves)]), *cache]
    parents, new = s["parents"].tolist(), s["new"].tolist()
    held = [tables[p][:count(lens[p])] if p >= 0 else [] for p in parents]
    for b in range(rows):
        for p in held[b]:
            refs[p] += 1
        for p in tables[b][:count(lens[b])]:
            refs[p] -= 1
    lens = [lens[p] if p >= 0 else 0 for p in parents]
    writers = {}
    for b in range(rows):
        if new[b] and lens[b] % page and refs[held[b][-1]] > 1:
            writers.setdefault(held[b][-1], []).append(b)
    copying = set()
    for p, who in writers.items():
        copying.update(who[1:] if len(who) == refs[p] else who)
    free = [p for p in range(pages) if refs[p] == 0]
    pairs = [[-1, -1] for _ in range(rows)]
    for b in range(rows):
        if b in copying:
            src, dst = held[b][-1], free.pop(0)
            pairs[b], held[b][-1] = [src, dst], dst
            refs[src] -= 1
            refs[dst] = 1
            for t in cache:
                t[:, dst] = t[:, src]
        lens[b] += new[b]
        while len(held[b]) < count(lens[b]):
            held[b].append(free.pop(0))
            refs[held[b][-1]] = 1
    tables = [h + [-1] * (width - len(h)) for h in held]
    return [_ints(tables), _ints(lens), _ints(refs), _ints(pairs), _ints([0, 0]), *cache]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rotate(s["x"], s["positions"], s["inv_freq"], s["magnitude"], case["layout"])
    if case["op"] == "append":
        return _exact_append(s, case)
    return _exact_attend(s, case) if case["op"] == "attend" else _exact_pages(s, case)
