"""A tree over a route made from its first tokens' queries, behind an append of the whole tree
(bounds: test_tree.py)."""

import pytest
import torch

from cache_helpers import dev
from helpers import lib
from test_tree import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return lib()


@pytest.mark.parametrize("budget", [4, 100])
@pytest.mark.parametrize("H,Hkv,S", [(8, 2, 3), (24, 2, 9)])
def test_by_the_first_tokens_queries(sa, H, Hkv, S, budget):
    lens = [1500, 640, 70, 0, 64]
    c = Case(lens, S, H, Hkv, 64, "bf16", seed=S)
    # sums as appends leave them: those of the page in progress with the drafts' keys
    k_sum = torch.nan_to_num(c.kc.float(), posinf=0.0).sum(2).contiguous()
    q = c.q.cuda()
    row_ptr, cols = sa.sa_route_pages(q[:, :1], k_sum, dev(c.table), dev(lens), 100, budget)
    rp, ci = row_ptr.tolist(), cols.tolist()
    rows = [ci[rp[i]:rp[i + 1]] for i in range(len(lens) * Hkv)]
    for i, r in enumerate(rows):
        full = lens[i // Hkv] // 64
        assert len(r) == min(-(-lens[i // Hkv] // 64), budget) and r == sorted(set(r))
        assert budget == 4 or set(range(full)) <= set(r)
    o, lse = c.run(sa, row_ptr=row_ptr, col_idx=cols)
    assert int(c.st.item()) == 0
    c.check(o, lse, rows)
    if budget == 100:                       # every page: as without a route
        o, lse = o.clone(), lse.clone()
        c.run(sa)
        c.check(o, lse)
