"""A row's bits come from its own query and what it sees: rows beside it in the same call change nothing."""
import pytest

import weight_only_quantization_pack_amd as awq

from cache_util import Case
from gpu_util import announce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("pairs,heads,kv,dim,page", [([(1, 900), (1, 40)], 16, 2, 64, 16), ([(7, 1500)], 8, 2, 128, 64),
                                                     ([(40, 700)], 4, 2, 64, 32), ([(150, 900), (90, 20)], 4, 2, 128, 64),
                                                     ([(120, 500)], 4, 2, 192, 16)], ids=str)
def test_other_rows_change_nothing(gpu, pairs, heads, kv, dim, page, window):
    """Queries of other rows and heads get other sizes, so that their maxima rise elsewhere."""
    import torch
    announce("attention neighbours", pairs, heads, kv, dim, page, window)
    case = Case(pairs, heads, kv, dim, page, seed=dim + page)
    cache, tables, lens, st = case.on_gpu()
    q = case.rows(heads, 4.0)

    def run(q):
        lse = torch.empty(case.T, heads, device="cuda")
        return awq.cache_attention(q, cache, tables, lens, st, window=window, max_new=max(case.new), lse=lse), lse

    want, want_lse = run(q)
    g = torch.Generator(device="cuda").manual_seed(page)
    for turn in range(4):
        keep = torch.rand(case.T, heads, device="cuda", generator=g) < 0.5
        sizes = torch.exp2(8.0 * torch.rand(case.T, heads, 1, device="cuda", generator=g) - 4.0)
        got, lse = run(torch.where(keep[..., None], q, (q.float() * sizes).to(q.dtype)))
        assert torch.equal(got[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])
