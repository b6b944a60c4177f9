"""GPU parity of awq_moe against the 64-bit layer on the oracle's dequantized
weights.

Bound.  All products take exact (q - z) codes, sums are fp32 and h keeps 22
bits, so before its one rounding y is off by fp32 sums: K and I values summed
in at most K / 128 + 40 dependent fp32 steps, (220 + 40) * 2^-24 < 2^-15 of the
sum of magnitudes in the worst order, of which random signs leave far less.
The bound is |y - ref| <= 2^-11 |ref| + 2^-13 max_k |ref[m]| per element: one
rounding, and 2^-13 of the row's largest value for the fp32 sums behind SiLU
and two products.  The inputs keep the top_k gap of the logits above 1e-3.
"""
import numpy as np
import pytest

import oracle as O
import weight_only_quantization_pack_amd as awq

import block_reference as R
from gpu_util import announce, dev, guarded_empty, host, sentinel_intact

pytestmark = pytest.mark.gpu


def experts(E, N, K, bits, group_size, seed):
    """(packed GPU tensors stacked over the experts, dequantized float64 layers)."""
    import torch
    g = np.random.default_rng(seed)
    packed, plain = [], []
    for _ in range(E):
        W = (0.05 * g.standard_normal((N, K))).astype(np.float16)
        q, d, z = O.quantize(W, None, bits, group_size)
        packed.append((dev(O.pack(q, bits).reshape(-1)), dev(O.tile_params(d)), dev(O.tile_params(z))))
        d64, z64 = (np.repeat(np.asarray(v, dtype=np.float64), group_size, axis=1) for v in (d, z))
        plain.append((q.astype(np.float64) - z64) * d64)
    return tuple(torch.stack(t) for t in zip(*packed)), plain


class Layer:
    def __init__(self, E, K, I, bits, group_size, seed=0):
        self.E, self.K, self.I, self.bits, self.group_size = E, K, I, bits, group_size
        self.gate, self.gate64 = experts(E, I, K, bits, group_size, seed + 1)
        self.up, self.up64 = experts(E, I, K, bits, group_size, seed + 2)
        self.down, self.down64 = experts(E, K, I, bits, group_size, seed + 3)

    def run(self, x, router, top_k, **kw):
        return awq.moe(x, router, self.gate, self.up, self.down, inter=self.I, top_k=top_k, bits=self.bits,
                       group_size=self.group_size, **kw)

    def ref(self, x, router, top_k, renormalize=True, inv_s=None):
        return R.moe(R.to_f64(x), R.to_f64(router), self.gate64, self.up64, self.down64, top_k, renormalize,
                     None if inv_s is None else R.to_f64(inv_s))


def router_of(E, K, x, top_k, seed):
    """Router weights whose logits on x have a gap at top_k."""
    import torch
    for s in range(seed, seed + 2000):
        g = np.random.default_rng(s)
        r = torch.from_numpy((2.0 / np.sqrt(K) * g.standard_normal((E, K))).astype(np.float16))
        if top_k == E:
            return r.cuda()
        l = np.sort(R.to_f64(x) @ R.to_f64(r).T, axis=1)[:, ::-1]
        if np.min(l[:, top_k - 1] - l[:, top_k]) > 1e-3:
            return r.cuda()
    raise AssertionError("no router with a gap")


def tokens(M, K, seed, shared=0.0):
    import torch
    g = np.random.default_rng(seed)
    x = (1 - shared) * g.standard_normal((M, K)) + shared * g.standard_normal((1, K))
    return torch.from_numpy(x.astype(np.float16)).cuda()


def check(y, ref):
    assert np.isfinite(ref).all()
    bound = 2.0 ** -11 * np.abs(ref) + 2.0 ** -13 * np.abs(ref).max(1, keepdims=True) + 2.0 ** -24
    worst = np.max(np.abs(R.to_f64(y) - ref) / bound)
    assert worst <= 1.0, f"{worst:.3f} of the bound"


# (M, E, top_k, K, I): one token, one expert, all experts, odd token counts and expert counts, more tokens than an
# operand tile, one k tile, tile counts that no wave count divides
SHAPES = [(1, 1, 1, 128, 128), (1, 8, 2, 512, 256), (1, 5, 5, 256, 384), (2, 7, 3, 384, 640), (5, 4, 2, 1024, 128),
          (9, 3, 1, 128, 1152), (13, 16, 6, 640, 384), (17, 4, 3, 512, 512), (33, 2, 1, 256, 256),
          (64, 6, 2, 384, 256), (64, 3, 3, 256, 128), (3, 70, 8, 256, 128)]


@pytest.mark.parametrize("bits", [4, 3])
@pytest.mark.parametrize("group_size", [128, 64])
@pytest.mark.parametrize("M,E,top_k,K,I", SHAPES)
def test_moe(gpu, M, E, top_k, K, I, group_size, bits):
    import torch
    announce("moe", f"M={M} E={E} top_k={top_k} K={K} I={I} bits={bits} gs={group_size}")
    layer = Layer(E, K, I, bits, group_size)
    x = tokens(M, K, 5)
    router = router_of(E, K, x, top_k, 6)
    g = np.random.default_rng(7)
    inv_s = dev(np.exp(0.3 * g.standard_normal(K)).astype(np.float32))
    for renorm, scale in ((True, None), (False, inv_s)):
        y, raw, n = guarded_empty((M, K), torch.float16)
        layer.run(x, router, top_k, renormalize=renorm, inv_s=scale, out=y)
        torch.cuda.synchronize()
        assert sentinel_intact(raw, n)
        check(y, layer.ref(x, router, top_k, renorm, scale))


@pytest.mark.parametrize("M,E,top_k,K,I", [(1, 4, 2, 4096, 1408), (16, 4, 2, 1408, 4096), (7, 3, 2, 512, 11008)])
def test_moe_long_rows(gpu, M, E, top_k, K, I):
    """Rows long enough for every wave count, and more tiles than waves."""
    announce("moe long", f"M={M} E={E} top_k={top_k} K={K} I={I}")
    layer = Layer(E, K, I, 4, 128)
    x = tokens(M, K, 5)
    router = router_of(E, K, x, top_k, 6)
    check(layer.run(x, router, top_k), layer.ref(x, router, top_k))


@pytest.mark.parametrize("bits", [4, 3])
@pytest.mark.parametrize("M,E,top_k,K,I", [(64, 8, 2, 2048, 2176), (31, 7, 4, 640, 3712)])
def test_moe_batches(gpu, M, E, top_k, K, I, bits):
    """Operands of 64 rows with a workgroup of 8 waves for half of the compute units or more, and with few
    workgroups whose K is split."""
    announce("moe batches", f"M={M} E={E} top_k={top_k} K={K} I={I} bits={bits}")
    layer = Layer(E, K, I, bits, 128)
    x = tokens(M, K, 5)
    router = router_of(E, K, x, top_k, 6)
    inv_s = dev(np.exp(0.3 * np.random.default_rng(7).standard_normal(K)).astype(np.float32))
    for scale in (None, inv_s):
        check(layer.run(x, router, top_k, inv_s=scale), layer.ref(x, router, top_k, True, scale))


@pytest.mark.parametrize("bits", [4, 3])
@pytest.mark.parametrize("group_size", [128, 64])
@pytest.mark.parametrize("M,E,top_k,K,I", [(2, 9, 1, 1024, 128), (13, 6, 2, 1152, 384), (40, 5, 2, 1408, 256),
                                           (64, 3, 3, 1664, 128)])
def test_moe_few_row_blocks(gpu, M, E, top_k, K, I, group_size, bits):
    """Gate and up projections whose row blocks are too few for the card: K in turns, with ragged last turns
    and experts that take several passes."""
    announce("moe few row blocks", f"M={M} E={E} top_k={top_k} K={K} I={I} bits={bits} gs={group_size}")
    layer = Layer(E, K, I, bits, group_size)
    x = tokens(M, K, 5)
    router = router_of(E, K, x, top_k, 6)
    inv_s = dev(np.exp(0.3 * np.random.default_rng(7).standard_normal(K)).astype(np.float32))
    for scale in (None, inv_s):
        check(layer.run(x, router, top_k, inv_s=scale), layer.ref(x, router, top_k, True, scale))


@pytest.mark.parametrize("group_size", [128, 64])
def test_every_token_on_the_same_experts(gpu, group_size):
    """All tokens choose the same experts of many: the others get no token."""
    layer = Layer(24, 256, 256, 4, group_size)
    x = tokens(64, 256, 5, shared=0.98)
    router = router_of(24, 256, x, 2, 6)
    ids, _ = R.route(R.to_f64(x) @ R.to_f64(router).T, 2, True)
    assert len(np.unique(ids)) <= 4
    check(layer.run(x, router, 2), layer.ref(x, router, 2))


def test_ties_go_to_the_lowest_index(gpu):
    """Equal logits (equal router rows, a zero row of x): the lowest experts."""
    import torch
    layer = Layer(70, 128, 128, 4, 128)
    x = tokens(3, 128, 5)
    x[1] = 0
    router = torch.zeros(70, 128, dtype=torch.float16, device="cuda")
    router[[9, 66, 40]] = tokens(1, 128, 8)
    router[5] = -router[9]
    check(layer.run(x, router, 2), layer.ref(x, router, 2))
    check(layer.run(x, router, 5, renormalize=False), layer.ref(x, router, 5, False))


def test_bad_tokens_stay_in_their_row(gpu):
    """NaN and infinite tokens route somewhere, and change no other token."""
    import torch
    layer = Layer(6, 256, 128, 4, 64)
    x = tokens(8, 256, 5)
    router = router_of(6, 256, x, 2, 6)
    y0 = layer.run(x, router, 2)
    x[2, 3] = float("nan")
    x[5, 9] = float("inf")
    y = layer.run(x, router, 2)
    torch.cuda.synchronize()
    keep = [0, 1, 3, 4, 6, 7]
    assert torch.equal(y[keep].view(torch.int16), y0[keep].view(torch.int16))
    assert not torch.isfinite(y[2]).any() and not torch.isfinite(y[5]).any()


def test_same_bits_again_on_another_stream_and_workspace(gpu):
    import torch
    layer = Layer(8, 512, 384, 4, 128)
    x = tokens(11, 512, 5)
    router = router_of(8, 512, x, 3, 6)
    y0 = layer.run(x, router, 3)
    need = awq.moe_workspace_bytes(11, 512, 384, 8, 3)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        ys = [layer.run(x, router, 3, workspace=ws) for _ in range(5)]
    st.synchronize()
    for y in ys:
        assert torch.equal(y.view(torch.int16), y0.view(torch.int16))
    with pytest.raises(awq.AwqError):
        layer.run(x, router, 3, workspace=ws[: need - 16])


def test_graph_replays(gpu):
    """Captured once, replayed with new tokens between eager calls."""
    import torch
    layer = Layer(8, 512, 384, 4, 128)
    x = tokens(3, 512, 5)
    router = router_of(8, 512, x, 2, 6)
    out = torch.empty_like(x)
    ws = torch.empty(awq.moe_workspace_bytes(3, 512, 384, 8, 2), dtype=torch.uint8, device="cuda")
    layer.run(x, router, 2, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.run(x, router, 2, out=out, workspace=ws)
    for seed in (5, 21, 22, 23):
        x.copy_(tokens(3, 512, seed))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        eager = layer.run(x, router, 2)
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), eager.view(torch.int16))


def test_refusals(gpu):
    import torch
    layer = Layer(4, 256, 128, 4, 128)
    x = tokens(4, 256, 5)
    router = router_of(4, 256, x, 2, 6)
    with pytest.raises(TypeError):
        layer.run(x.bfloat16(), router, 2)
    with pytest.raises(TypeError):
        layer.run(x, router.float(), 2)
    with pytest.raises(ValueError):
        layer.run(x, router[:3], 2)
    with pytest.raises(ValueError):
        layer.run(x[:, :128], router, 2)
    with pytest.raises(ValueError):
        awq.moe(x, router, layer.gate, layer.up, layer.gate, inter=128, top_k=2)
    with pytest.raises(ValueError):
        layer.run(x, router, 2, inv_s=torch.ones(128, device="cuda"))
    for top_k in (0, 5):
        with pytest.raises(awq.AwqError):
            layer.run(x, router, top_k)
    with pytest.raises(awq.AwqError):
        layer.run(tokens(65, 256, 1), router, 2)
    assert layer.run(x[:0], router, 2).shape == (0, 256)
