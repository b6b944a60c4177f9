"""A layer's slice of a cache of several layers in every call that takes one."""
import pytest

import weight_only_quantization_pack_amd as awq

from cache_util import ints
from gpu_util import announce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv,pages", [(1, 7), (2, 5), (3, 9), (4, 6), (8, 4)])
def test_copies_in_one_layer(gpu, kv, pages):
    """Scales of a layer begin at any word of 4 bytes; the other layers stay as they are."""
    import torch
    announce("copy in a layer", kv, pages)
    layers, page, dim = 3, 16, 64
    cache = awq.empty_cache(pages, kv, page, dim, layers=layers)
    g = torch.Generator(device="cuda").manual_seed(kv)
    for t in cache:
        t.copy_(torch.randint(-127, 128, t.shape, device="cuda", generator=g))
    pairs = ints([[0, pages - 1], [-1, -1], [2, 1]])
    for layer in range(layers):
        want = [t.clone() for t in cache]
        for t in want:
            t[layer, pages - 1] = t[layer, 0]
            t[layer, 1] = t[layer, 2]
        awq.cache_copy_pages([t[layer] for t in cache], pairs)
        for t, w in zip(cache, want):
            assert torch.equal(t, w)
