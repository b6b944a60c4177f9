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


@pytest.mark.parametrize("pairs,heads,kv,dim", [([(100, 20000)], 8, 1, 64), ([(64, 9000), (40, 30000)], 16, 2, 128),
                                                ([(40, 30000)], 4, 1, 256)], ids=str)
def test_short_windows_leave_no_parts(gpu, pairs, heads, kv, dim):
    """A tile whose rows see two or three tiles of keys is not split, however long the sequence: nothing goes through the
    workspace, and the bound that its size comes from still does where there is no window."""
    import torch
    announce("attention short windows", pairs, heads, kv, dim)
    case = Case(pairs, heads, kv, dim, 64, seed=dim)
    cache, tables, lens, st = case.on_gpu()
    q = case.rows(heads, 2.0)
    most = max(n + p for n, p in pairs)
    bounds = dict(max_new=max(case.new), max_len=most)
    need = awq.cache_attention_workspace_bytes(case.T, len(pairs), heads, kv, dim, max(case.new), most)
    assert need > 0
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")
    got = awq.cache_attention(q, cache, tables, lens, st, window=32, workspace=ws, **bounds)
    torch.cuda.synchronize()
    assert bool((ws == 0xA5).all())
    # the same rows over the same keys, in a call that knows only short sequences
    want = awq.cache_attention(q, cache, tables, lens, st, window=32, max_new=max(case.new), max_len=64)
    assert torch.equal(got, want)
    awq.cache_attention(q, cache, tables, lens, st, workspace=ws, **bounds)
    torch.cuda.synchronize()
    assert not bool((ws == 0xA5).all())
