"""awq_moe over the ends of its range, and every way in which one token's
products are cut.

Bounds and references as in test_gpu_moe.py, whose bound of 2^-15 for fp32 sums
holds up to the longest rows: K / 128 + 40 = 296 dependent steps of 2^-24.  Many
experts share a few different weights (expert e holds those of e % distinct), so
that the oracle's packing stays short.
"""
import numpy as np
import pytest

import oracle as O
import weight_only_quantization_pack_amd as awq

import block_reference as R
from gpu_util import announce, dev, guarded_empty, sentinel_intact
from test_gpu_moe import Layer, check, router_of, tokens

pytestmark = pytest.mark.gpu


class SharedLayer(Layer):
    """E experts of `distinct` different weights of the given size."""

    def __init__(self, E, K, I, bits, group_size, distinct=3, size=0.05):
        import torch
        self.E, self.K, self.I, self.bits, self.group_size = E, K, I, bits, group_size
        pick = torch.arange(E, device="cuda") % distinct

        def experts(N, Kin, seed):
            g = np.random.default_rng(seed)
            packed, plain = [], []
            for _ in range(min(E, distinct)):
                W = (size * g.standard_normal((N, Kin))).astype(np.float16)
                q, d, z = O.quantize(W, None, bits, group_size)
                packed.append((dev(O.pack(q, bits).reshape(-1)), dev(O.tile_params(d)), dev(O.tile_params(z))))
                d64, z64 = (np.repeat(np.asarray(v, dtype=np.float64), group_size, axis=1) for v in (d, z))
                plain.append((q.astype(np.float64) - z64) * d64)
            return (tuple(torch.stack(t)[pick].contiguous() for t in zip(*packed)),
                    [plain[e % distinct] for e in range(E)])
        self.gate, self.gate64 = experts(I, K, 1)
        self.up, self.up64 = experts(I, K, 2)
        self.down, self.down64 = experts(K, I, 3)


def scale_of(K):
    return dev(np.exp(0.3 * np.random.default_rng(7).standard_normal(K)).astype(np.float32))


# K / 128 and I / 128 on both sides of 8 and 32 tiles (2, 4 and 8 waves of an item), ragged last turns of the waves
@pytest.mark.parametrize("bits", [4, 3])
@pytest.mark.parametrize("group_size", [128, 64])
@pytest.mark.parametrize("E,top_k,K,I", [(4, 3, 896, 1024), (4, 3, 1024, 4096), (4, 2, 3968, 1152), (3, 2, 4096, 896),
                                         (4, 1, 1408, 4224), (3, 3, 4224, 3968)])
def test_one_token(gpu, E, top_k, K, I, group_size, bits):
    import torch
    announce("moe one token", f"E={E} top_k={top_k} K={K} I={I} bits={bits} gs={group_size}")
    layer = SharedLayer(E, K, I, bits, group_size)
    x = tokens(1, K, 5)
    router = router_of(E, K, x, top_k, 6)
    for renorm, scale in ((True, None), (False, scale_of(K))):
        y, raw, n = guarded_empty((1, K), torch.float16)
        layer.run(x, router, top_k, renormalize=renorm, inv_s=scale, out=y)
        torch.cuda.synchronize()
        assert sentinel_intact(raw, n)
        check(y, layer.ref(x, router, top_k, renorm, scale))


# operands of one token past 48 KB of LDS (both products), and 4 to 16 parts of the router's rows
@pytest.mark.parametrize("M,E,top_k,K,I", [(1, 4, 2, 256, 14336), (1, 3, 2, 14336, 256), (1, 64, 8, 6272, 128),
                                           (1, 3, 1, 128, 32768), (1, 512, 16, 32768, 128), (6, 3, 2, 32768, 256),
                                           (3, 4, 2, 128, 32768), (9, 512, 16, 6272, 128), (64, 512, 16, 128, 256),
                                           (64, 20, 16, 256, 128)])
@pytest.mark.parametrize("bits,group_size", [(4, 128), (3, 64)])
def test_ends_of_the_range(gpu, M, E, top_k, K, I, bits, group_size):
    announce("moe range", f"M={M} E={E} top_k={top_k} K={K} I={I} bits={bits} gs={group_size}")
    layer = SharedLayer(E, K, I, bits, group_size)
    x = tokens(M, K, 5)
    router = router_of(E, K, x, top_k, 6)
    for scale in (None, scale_of(K)):
        check(layer.run(x, router, top_k, inv_s=scale), layer.ref(x, router, top_k, True, scale))


@pytest.mark.parametrize("top_k", [1, 2, 5, 8, 16])
def test_one_token_same_bits_on_another_stream_and_workspace(gpu, top_k):
    """The exchange inside one token's down product: a workspace of any contents, calls one after another."""
    import torch
    layer = SharedLayer(17, 1024, 512, 4, 128, distinct=5)
    x = tokens(1, 1024, 5)
    router = router_of(17, 1024, x, top_k, 6)
    y0 = layer.run(x, router, top_k)
    check(y0, layer.ref(x, router, top_k))
    ws = torch.full((awq.moe_workspace_bytes(1, 1024, 512, 17, top_k),), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        ys = [layer.run(x, router, top_k, workspace=ws) for _ in range(20)]
    st.synchronize()
    for y in ys:
        assert torch.equal(y.view(torch.int16), y0.view(torch.int16))


@pytest.mark.parametrize("M,top_k", [(1, 2), (1, 8), (2, 8)])
def test_graph_replays_of_few_tokens(gpu, M, top_k):
    """Captured once, replayed with new tokens between eager calls."""
    import torch
    layer = SharedLayer(12, 512, 1024, 4, 64, distinct=5)
    x = tokens(M, 512, 5)
    router = router_of(12, 512, x, top_k, 6)
    out = torch.empty_like(x)
    ws = torch.empty(awq.moe_workspace_bytes(M, 512, 1024, 12, top_k), dtype=torch.uint8, device="cuda")
    layer.run(x, router, top_k, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.run(x, router, top_k, out=out, workspace=ws)
    for seed in (5, 21, 22, 23, 24):
        x.copy_(tokens(M, 512, seed))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        eager = layer.run(x, router, top_k)
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), eager.view(torch.int16))


def test_router_weights_below_the_normal_fp16_range(gpu):
    """fp16 subnormals in the router choose as their values say."""
    import torch
    layer = SharedLayer(8, 512, 128, 4, 128)
    g = np.random.default_rng(1)
    x = torch.from_numpy((300 * g.standard_normal((4, 512))).astype(np.float16)).cuda()
    router = torch.from_numpy((2.0 ** -17 * g.standard_normal((8, 512))).astype(np.float16)).cuda()
    logits = np.sort(R.to_f64(x) @ R.to_f64(router).T, axis=1)
    assert np.min(logits[:, -2] - logits[:, -3]) > 1e-3
    for rows in (slice(0, 1), slice(0, 4)):
        # x / 300: the same choices from logits 300 times smaller, fp32 sums of gaps above 3e-6
        check(layer.run(x[rows] / 300, router, 2), layer.ref(x[rows] / 300, router, 2))


@pytest.mark.parametrize("M", [1, 3])
def test_scaled_tokens_up_to_the_fp16_maximum(gpu, M):
    """x * inv_s of 60000 is exact to 22 bits like any other; past the fp16 maximum its token's row is NaN and no
    other token changes."""
    import torch
    layer = SharedLayer(5, 256, 128, 4, 128, size=5e-4)
    x = tokens(M, 256, 5)
    inv_s = torch.ones(256, device="cuda")
    inv_s[7] = 100.0
    x[0, 7] = 600.0
    router = router_of(5, 256, x, 2, 6)
    router[:, 7] = 0
    logits = np.sort(R.to_f64(x) @ R.to_f64(router).T, axis=1)
    assert np.min(logits[:, -2] - logits[:, -3]) > 1e-3
    y0 = layer.run(x, router, 2, inv_s=inv_s)
    check(y0, layer.ref(x, router, 2, True, inv_s))
    x[0, 7] = 700.0
    y = layer.run(x, router, 2, inv_s=inv_s)
    assert torch.isnan(y[0]).all() and torch.equal(y[1:].view(torch.int16), y0[1:].view(torch.int16))


@pytest.mark.parametrize("M", [1, 3])
def test_gated_values_past_the_fp16_maximum(gpu, M):
    """SiLU(gate) * up past the fp16 maximum: a row of NaN, and no other token changes."""
    import torch
    layer = SharedLayer(5, 256, 128, 4, 64)
    x = tokens(M, 256, 5)
    router = router_of(5, 256, x, 2, 6)
    y0 = layer.run(x, router, 2)
    x[0] *= 2000
    y = layer.run(x, router, 2)
    assert torch.isnan(y[0]).all() and torch.equal(y[1:].view(torch.int16), y0[1:].view(torch.int16))
