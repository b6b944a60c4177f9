"""Windows of attention: how large they may be, and what short ones cost behind long sequences."""
import pytest

import weight_only_quantization_pack_amd as awq

from cache_util import Case
from gpu_util import announce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pairs", [[(1, 300)], [(90, 200)]], ids=str)
def test_windows_past_31_bits(gpu, pairs):
    """Any window as long as the sequence is none, also where a C int would wrap around; negative ones are refused."""
    import torch
    announce("attention wide windows", pairs)
    case = Case(pairs, 4, 2, 64, 16, seed=1)
    cache, tables, lens, st = case.on_gpu()
    q = case.rows(4, 2.0)
    want = awq.cache_attention(q, cache, tables, lens, st)
    for window in (1 << 30, (1 << 31) - 1, 1 << 31, (1 << 32) + 5, (1 << 63) + 5):
        assert torch.equal(awq.cache_attention(q, cache, tables, lens, st, window=window), want), window
    for window in (-1, -(1 << 31), -(1 << 32), -(1 << 32) + 5):
        with pytest.raises(awq.AwqError):
            awq.cache_attention(q, cache, tables, lens, st, window=window)
