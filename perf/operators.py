"""Cases of the operators that stand beside the packed W4A16 / W3A16 products in a decoder block.

Three operators, each with its cases, its inputs, its plain form and its 64-bit definition:

  norm   the norm after a block, its gate, the scaled residual and the norm before the next block:
             t  = post(b)                (RMS or layer norm; t = b without one)
             r' = alpha * r + g * t
             h  = pre(r')                (from r' before it is rounded for storage)
  w8a8   a product in 8-bit integers with one scale for each token and each channel:
             y[m][n] = sx[m] * sw[n] * sum_k xq[m][k] * wq[n][k]  (+ bias[n])
         where the activations come as codes ("int8"), as 16-bit rows that the call quantizes
         (sx = max|x| / 127, xq = rint(127 x / max|x|): "rows"), or as the norm above writes them ("norm").
  moe    a mixture-of-experts layer for a few tokens over packed experts:
             l = x Wr^T;  the top_k largest l of each token (ties to the lowest index);
             p = softmax(l) over the chosen ones (renormalize) or over all experts;
             y = sum_j p_j down_j(SiLU(gate_j x) * up_j x)
         with the experts in the library's packed format 3.

`run` takes what `prepare` gives through the plain form (elementary torch operations in 32 bits,
rounded once) where `own` is false, and through the library's entry points where it is true.
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
        # one token between two blocks of a 4096-wide decoder: launch latency is the whole cost
        dict(name="norm_one_token", op="norm", tokens=1, width=4096, dtype="fp16", kind="rms",
             post=True, gate=0, alpha=1.0),
        # a decode batch with a learned gate per channel
        dict(name="norm_batch", op="norm", tokens=64, width=8192, dtype="bf16", kind="rms",
             post=True, gate=1, alpha=1.0),
        # an ordinary prompt, the residual scaled by the depth, no norm after the block
        dict(name="norm_prompt", op="norm", tokens=2048, width=4096, dtype="fp16", kind="rms",
             post=False, gate=0, alpha=0.7),
        # a long odd prompt of three conditioned sequences: layer norms and one gate row for each sequence
        dict(name="norm_conditioned", op="norm", tokens=8193, width=8192, dtype="bf16", kind="layer",
             post=True, gate=3, alpha=1.0),
        # one token through a wide projection: the weight read is the cost
        dict(name="w8a8_one_token", op="w8a8", tokens=1, width=4096, out=11008, dtype="fp16",
             source="rows", bias=False),
        # a decode batch through the widest projection, behind the norm that writes its codes
        dict(name="w8a8_batch", op="w8a8", tokens=16, width=8192, out=28672, dtype="bf16",
             source="norm", bias=False),
        # a ragged prompt chunk into a fused q/k/v projection with a bias
        dict(name="w8a8_chunk", op="w8a8", tokens=509, width=4096, out=6144, dtype="fp16",
             source="rows", bias=True),
        # a long prompt through an MLP projection, codes in hand: the matrix pipes are the cost
        dict(name="w8a8_prompt", op="w8a8", tokens=8192, width=4096, out=14336, dtype="bf16",
             source="int8", bias=False),
        # one token, many narrow experts: launches and latency
        dict(name="moe_one_token_narrow", op="moe", tokens=1, width=2048, inter=768, experts=128, top_k=8,
             bits=4, group=128, renorm=True, scaled=False),
        # one token, few wide experts: the weight read is the cost
        dict(name="moe_one_token_wide", op="moe", tokens=1, width=4096, inter=14336, experts=8, top_k=2,
             bits=4, group=128, renorm=True, scaled=False),
        # a decode batch of odd size over 3-bit experts with 64-wide groups and an activation scale
        dict(name="moe_batch_int3", op="moe", tokens=13, width=2048, inter=1408, experts=64, top_k=6,
             bits=3, group=64, renorm=False, scaled=True),
        # a full decode batch that reaches every wide expert
        dict(name="moe_batch_wide", op="moe", tokens=64, width=4096, inter=14336, experts=8, top_k=2,
             bits=4, group=128, renorm=True, scaled=False),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in lo..hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return min(hi, max(lo, int(v) // step * step))


def draw(rng):
    op = rng.choice(["norm", "w8a8", "moe"])
    if op == "norm":
        tokens = _log(rng, 1, 8192)
        groups = rng.choice([0, 1, 1, 4])
        if groups == 4:
            tokens = max(4, tokens // 4 * 4)
        return dict(op=op, tokens=tokens, width=_log(rng, 256, 8192, 8), dtype=rng.choice(["fp16", "bf16"]),
                    kind=rng.choice(["rms", "layer"]), post=rng.random() < 0.6, gate=groups,
                    alpha=rng.choice([1.0, 0.7, 1.25]))
    if op == "w8a8":
        width, out = _log(rng, 256, 28672, 16), _log(rng, 64, 28672)
        most = 8192 * 4096 * 14336 // (width * out)
        return dict(op=op, tokens=_log(rng, 1, max(1, min(8192, most))), width=width, out=out,
                    dtype=rng.choice(["fp16", "bf16"]), source=rng.choice(["rows", "norm", "int8"]),
                    bias=rng.random() < 0.4)
    experts = _log(rng, 4, 128)
    width, inter = _log(rng, 512, 4096, 128), _log(rng, 256, 14336, 128)
    while experts * width * inter > 8 * 4096 * 14336:
        experts, inter = max(4, experts // 2), max(256, inter // 256 * 128)
    return dict(op=op, tokens=_log(rng, 1, 64), width=width, inter=inter, experts=experts,
                top_k=rng.randint(1, min(8, experts)), bits=rng.choice([4, 4, 3]), group=rng.choice([128, 64]),
                renorm=rng.random() < 0.5, scaled=rng.random() < 0.3)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device=DEV)


def _activations(g, tokens, width):
    """Rows whose channels differ in size, as they do behind a decoder block."""
    return _randn(g, tokens, width) * torch.exp(0.6 * _randn(g, width))


def _norm_state(g, c, dtype):
    t, w = c["tokens"], c["width"]
    s = dict(block=_activations(g, t, w).to(dtype), residual=(4.0 * _activations(g, t, w)).to(dtype),
             pre_weight=(1.0 + 0.2 * _randn(g, w)).to(dtype), post_weight=None, pre_bias=None, post_bias=None,
             gate=None)
    if c["kind"] == "layer":
        s["pre_bias"] = (0.1 * _randn(g, w)).to(dtype)
    if c["post"]:
        s["post_weight"] = (0.5 + 0.1 * _randn(g, w)).to(dtype)
        if c["kind"] == "layer":
            s["post_bias"] = (0.1 * _randn(g, w)).to(dtype)
    if c["gate"]:
        s["gate"] = torch.tanh(_randn(g, c["gate"], w)).to(dtype)
    return s


# the norm in front of a "norm" product
PLAIN_NORM = dict(kind="rms", post=False, gate=0, alpha=1.0)

# bit position of code e of a packed int4 word
SHIFT4 = [4 * (e // 2) + 16 * (e % 2) for e in range(8)]


def _packed_codes(g, shape, bits):
    """Random codes around the middle of their range, already in packed order (the order does not
    matter for independent codes): int32 [shape][4 or 3]."""
    top = 2 ** bits - 1
    n = 8 if bits == 4 else 32
    words = 4 if bits == 4 else 1
    c = _randn(g, *shape, words, n).mul_(top / 5.8).add_(top / 2).round_().clamp_(0, top).to(torch.int32)
    if bits == 4:
        w = c[..., 0].clone()
        for e in range(1, 8):
            w |= c[..., e] << SHIFT4[e]
        return w
    c = c[..., 0, :]
    out = []
    for b in range(3):
        w = ((c[..., 30] >> b) & 1) << 15 | ((c[..., 31] >> b) & 1) << 31
        for p in range(5):
            pair = 5 * b + p
            w |= c[..., 2 * pair] << (3 * p) | c[..., 2 * pair + 1] << (16 + 3 * p)
        out.append(w)
    return torch.stack(out, dim=-1)


def _expert_layer(g, experts, rows, width, bits, group):
    """`experts` packed layers [rows][width]: qweight int32 [E][words], scales and zeros fp16 [E][rows/16][G][16]."""
    blocks, tiles, groups = (rows + 15) // 16, width // 128, width // group
    q = torch.stack([_packed_codes(g, (blocks, tiles, 64), bits).reshape(-1) for _ in range(experts)])
    top = 2 ** bits - 1
    d = (0.02 * 5.8 / top * (0.7 + 0.6 * _rand(g, experts, blocks, groups, 16))).to(torch.float16)
    z = (top / 2 + _randn(g, experts, blocks, groups, 16)).round_().clamp_(0, top).to(torch.float16)
    return q, d, z


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case=dict(c))
    if c["op"] == "norm":
        s.update(_norm_state(g, c, DTYPES[c["dtype"]]))
    elif c["op"] == "w8a8":
        dtype = DTYPES[c["dtype"]]
        t, k, n = c["tokens"], c["width"], c["out"]
        s["weight"] = _randn(g, n, k).mul_(32.0).round_().clamp_(-127, 127).to(torch.int8)
        s["weight_scales"] = 0.02 / 32.0 * torch.exp(0.3 * _randn(g, n))
        s["bias"] = _randn(g, n) if c["bias"] else None
        if c["source"] == "rows":
            s["x"] = _activations(g, t, k).to(dtype)
        elif c["source"] == "norm":
            s.update(_norm_state(g, dict(c, **PLAIN_NORM), dtype))
        else:
            s["q"] = _activations(g, t, k).mul_(12.0).round_().clamp_(-127, 127).to(torch.int8)
            s["q_scales"] = 0.05 * torch.exp(0.3 * _randn(g, t))
    else:
        t, k, i, e = c["tokens"], c["width"], c["inter"], c["experts"]
        # a part that all tokens share makes some experts more popular than others
        s["x"] = (_randn(g, t, k) + 0.5 * _randn(g, 1, k)).to(torch.float16)
        s["router"] = (2.0 / math.sqrt(k) * _randn(g, e, k)).to(torch.float16)
        s["inv_s"] = torch.exp(0.2 * _randn(g, k)) if c["scaled"] else None
        s["gate_proj"] = _expert_layer(g, e, i, k, c["bits"], c["group"])
        s["up_proj"] = _expert_layer(g, e, i, k, c["bits"], c["group"])
        s["down_proj"] = _expert_layer(g, e, k, i, c["bits"], c["group"])
    return s


# ---------------------------------------------------------------------------
# plain forms: 32 bits, one rounding at the end
# ---------------------------------------------------------------------------
EPS = 1e-6


def _plain_norm(v, weight, bias, kind):
    if kind == "layer":
        v = v - v.mean(dim=-1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(dim=-1, keepdim=True) + EPS) * weight.float()
    return v if bias is None else v + bias.float()


def _plain_norm_rows(s, c):
    """(r', h) in 32 bits."""
    t = s["block"].float()
    if s["post_weight"] is not None:
        t = _plain_norm(t, s["post_weight"], s["post_bias"], c["kind"])
    if s["gate"] is not None:
        n = s["gate"].shape[0]
        t = (t.reshape(n, -1, t.shape[-1]) * s["gate"].float()[:, None, :]).reshape(t.shape)
    r = c["alpha"] * s["residual"].float() + t
    return r, _plain_norm(r, s["pre_weight"], s["pre_bias"], c["kind"])


def _plain_quantize(x):
    """Codes (held as floats) and scales of the rows of x."""
    top = x.abs().amax(dim=-1, keepdim=True)
    return torch.where(top > 0, torch.round(x * 127.0 / top), torch.zeros_like(x)), top / 127.0


def _plain_w8a8(s, c):
    dtype = DTYPES[c["dtype"]]
    r = None
    if c["source"] == "int8":
        q, scale = s["q"].float(), s["q_scales"][:, None]
    elif c["source"] == "rows":
        q, scale = _plain_quantize(s["x"].float())
    else:
        r, h = _plain_norm_rows(s, dict(c, **PLAIN_NORM))
        q, scale = _plain_quantize(h)
    y = (q @ s["weight"].float().t()) * scale * s["weight_scales"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(dtype) if r is None else (r.to(dtype), y.to(dtype))


def _plain_unpack(layer, pick, width, bits, group):
    """Dequantized weights of the experts `pick`, 32 bits [len(pick)][rows][width]."""
    q, d, z = (v[pick] for v in layer)
    e, blocks, groups, _ = d.shape
    tiles = width // 128
    if bits == 4:
        shift = torch.tensor(SHIFT4, device=q.device, dtype=torch.int32)
        code = (q.reshape(e, blocks, tiles, 4, 16, 4, 1) >> shift) & 15
        code = code.reshape(e, blocks, tiles, 4, 16, 32)
    else:
        n = torch.arange(30, device=q.device)
        shift = (3 * (n // 2 % 5) + 16 * (n % 2)).to(torch.int32)
        w = q.reshape(e, blocks, tiles, 4, 16, 3)
        low = (w[..., n // 10] >> shift) & 7
        b = torch.arange(3, device=q.device, dtype=torch.int32)
        last = [(((w >> at) & 1) << b).sum(dim=-1, keepdim=True) for at in (15, 31)]
        code = torch.cat([low, *last], dim=-1)
    code = code.permute(0, 1, 4, 2, 3, 5).reshape(e, blocks * 16, groups, group).float()
    d, z = (v.permute(0, 1, 3, 2).reshape(e, blocks * 16, groups, 1).float() for v in (d, z))
    return ((code - z) * d).reshape(e, blocks * 16, width)


def _plain_moe(s, c):
    t, k, i, e, n = c["tokens"], c["width"], c["inter"], c["experts"], c["top_k"]
    x = s["x"].float()
    logits = x @ s["router"].float().t()
    order = torch.sort(logits, dim=-1, descending=True, stable=True)      # ties to the lowest index
    ids, chosen = order.indices[:, :n], order.values[:, :n]
    p = torch.exp(chosen - chosen[:, :1])
    p = p / (p if c["renorm"] else torch.exp(logits - chosen[:, :1])).sum(dim=-1, keepdim=True)
    if s["inv_s"] is not None:
        x = x * s["inv_s"]
    if t * n < e:             # few assignments: the weights of each one
        pick, rows = ids.reshape(-1), x.repeat_interleave(n, dim=0)[:, None, :]
        part = p.reshape(-1, 1, 1)
    else:                     # every expert over every token, weighted by its share (mostly zero)
        pick, rows = torch.arange(e, device=x.device), x[None].expand(e, t, k)
        part = torch.zeros(t, e, device=x.device).scatter_(1, ids, p).t()[:, :, None]
    gate = rows @ _plain_unpack(s["gate_proj"], pick, k, c["bits"], c["group"]).transpose(1, 2)
    up = rows @ _plain_unpack(s["up_proj"], pick, k, c["bits"], c["group"]).transpose(1, 2)
    h = gate / (1.0 + torch.exp(-gate)) * up
    y = (h @ _plain_unpack(s["down_proj"], pick, i, c["bits"], c["group"]).transpose(1, 2)) * part
    y = y.reshape(t, n, k).sum(dim=1) if t * n < e else y.sum(dim=0)
    return y.to(torch.float16)


def _plain(s, c):
    if c["op"] == "norm":
        r, h = _plain_norm_rows(s, c)
        return r.to(DTYPES[c["dtype"]]), h.to(DTYPES[c["dtype"]])
    return _plain_w8a8(s, c) if c["op"] == "w8a8" else _plain_moe(s, c)


# ---------------------------------------------------------------------------
# the library's operators
# ---------------------------------------------------------------------------
def _own(s, c):
    import weight_only_quantization_pack_amd as awq

    if c["op"] == "norm":
        return awq.norm_gate_residual(s["block"], s["residual"], s["pre_weight"], post_weight=s["post_weight"],
                                      gate=s["gate"], residual_scale=c["alpha"], kind=c["kind"],
                                      pre_bias=s["pre_bias"], post_bias=s["post_bias"], eps=EPS)
    if c["op"] == "w8a8":
        if c["source"] == "rows":
            return awq.linear_w8a8(s["x"], s["weight"], s["weight_scales"], bias=s["bias"])
        if c["source"] == "int8":
            return awq.gemm_w8a8(s["q"], s["q_scales"], s["weight"], s["weight_scales"], bias=s["bias"],
                                 dtype=DTYPES[c["dtype"]])
        r, q, scale = awq.norm_gate_residual(s["block"], s["residual"], s["pre_weight"], kind="rms", eps=EPS,
                                             quantize=True)
        return r, awq.gemm_w8a8(q, scale, s["weight"], s["weight_scales"], bias=s["bias"],
                                dtype=DTYPES[c["dtype"]])
    return awq.moe(s["x"], s["router"], s["gate_proj"], s["up_proj"], s["down_proj"], inter=c["inter"],
                   top_k=c["top_k"], bits=c["bits"], group_size=c["group"], renormalize=c["renorm"],
                   inv_s=s["inv_s"])


def run(state):
    return _own(state, state["case"]) if own else _plain(state, state["case"])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    t, k = c["tokens"], c["width"]
    if c["op"] == "norm":
        # block and residual in, residual and h out
        return {"bytes": 8 * t * k + 2 * k * (1 + c["post"] + c["gate"]), "flops": 12 * t * k}
    if c["op"] == "w8a8":
        n = c["out"]
        rows = {"int8": t * k, "rows": 2 * t * k, "norm": 6 * t * k}[c["source"]]
        return {"bytes": n * k + 4 * n + rows + 2 * t * n, "flops": 2 * t * n * k}
    i, e, top = c["inter"], c["experts"], c["top_k"]
    reached = e * (1.0 - (1.0 - top / e) ** t)            # experts that some token takes, on average
    weights = 3 * k * i * (c["bits"] / 8 + 4 / c["group"])
    return {"bytes": reached * weights + 2 * e * k + 4 * t * k, "flops": 6 * t * top * k * i + 2 * t * e * k}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_norm(s, c):
    def norm(v, w, b):
        if c["kind"] == "layer":
            centred = v - v.sum(-1, keepdim=True) / v.shape[-1]
        else:
            centred = v
        out = centred / (centred.pow(2).sum(-1, keepdim=True) / v.shape[-1] + EPS).sqrt() * w.double()
        return out + b.double() if b is not None else out

    out = s["block"].double()
    if s["post_weight"] is not None:
        out = norm(out, s["post_weight"], s["post_bias"])
    if s["gate"] is not None:
        each = out.shape[0] // s["gate"].shape[0]
        out = out * s["gate"].double()[torch.arange(out.shape[0], device=out.device) // each]
    r = s["residual"].double() * c["alpha"] + out
    return r, norm(r, s["pre_weight"], s["pre_bias"])


def _exact_codes(x):
    top = x.abs().max(dim=1).values
    safe = torch.where(top == 0, torch.ones_like(top), top)
    return (x * 127.0 / safe[:, None]).round(), top / 127.0


def _exact_w8a8(s, c):
    r = None
    if c["source"] == "int8":
        q, scale = s["q"].double(), s["q_scales"].double()
    elif c["source"] == "rows":
        q, scale = _exact_codes(s["x"].double())
    else:
        r, h = _exact_norm(s, dict(c, **PLAIN_NORM))
        q, scale = _exact_codes(h)
    y = torch.empty(c["tokens"], c["out"], dtype=torch.float64, device=DEV)
    for at in range(0, c["out"], 4096):                   # column by column block: 64-bit weights are wide
        w = s["weight"][at:at + 4096].double() * s["weight_scales"][at:at + 4096].double()[:, None]
        y[:, at:at + 4096] = (q @ w.t()) * scale[:, None]
    if s["bias"] is not None:
        y += s["bias"].double()
    return y if r is None else (r, y)


def _exact_layer(layer, e, rows, width, bits, group):
    """Expert e's dequantized weights in 64 bits, code by code from the format's description."""
    q = layer[0][e].reshape(-1, width // 128, 4, 16, 4 if bits == 4 else 3).long() & 0xFFFFFFFF
    code = torch.zeros(*q.shape[:-1], 32, dtype=torch.int64, device=q.device)
    for n in range(32):
        if bits == 4:
            code[..., n] = (q[..., n // 8] >> (4 * (n % 8 // 2) + 16 * (n % 2))) & 15
        elif n < 30:
            code[..., n] = (q[..., n // 2 // 5] >> (3 * (n // 2 % 5) + 16 * (n % 2))) & 7
        else:
            for b in range(3):
                code[..., n] += ((q[..., b] >> (15 if n == 30 else 31)) & 1) * 2 ** b
    code = code.permute(0, 3, 1, 2, 4).reshape(-1, width)[:rows].double()
    at = torch.arange(width, device=q.device) // group
    d, z = (v[e].permute(0, 2, 1).reshape(-1, width // group)[:rows].double()[:, at] for v in layer[1:])
    return (code - z) * d


def _exact_moe(s, c):
    x = s["x"].double()
    logits = x @ s["router"].double().t()
    left, ids = logits.clone(), []
    for _ in range(c["top_k"]):                           # one after the other: the lowest index among equals
        best = (left == left.max(dim=1, keepdim=True).values).long().argmax(dim=1)
        ids.append(best)
        left[torch.arange(len(best), device=DEV), best] = -math.inf
    chosen = torch.zeros_like(logits, dtype=torch.bool)
    for best in ids:
        chosen[torch.arange(len(best), device=DEV), best] = True
    weight = torch.softmax(logits.masked_fill(~chosen, -math.inf) if c["renorm"] else logits, dim=1)
    if s["inv_s"] is not None:
        x = x * s["inv_s"].double()
    y = torch.zeros_like(x)
    for e in range(c["experts"]):
        rows = chosen[:, e].nonzero()[:, 0]
        if not len(rows):
            continue
        gate, up, down = (_exact_layer(s[n], e, o, w, c["bits"], c["group"]) for n, o, w in (
            ("gate_proj", c["inter"], c["width"]), ("up_proj", c["inter"], c["width"]),
            ("down_proj", c["width"], c["inter"])))
        a = x[rows] @ gate.t()
        y[rows] += (a * torch.sigmoid(a) * (x[rows] @ up.t())) @ down.t() * weight[rows, e][:, None]
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s, case)
    return _exact_w8a8(s, case) if case["op"] == "w8a8" else _exact_moe(s, case)
