"""sa_route_pages where scores in fp64 differ, but by less than anything short of fp64
tells apart: the list is still that of the fp64 scores.

Every page of a row has the same sums but for one small element, whose product with the
query moves the score in steps of 2^-44, about 2^-50 of it. Products are multiples of 2^-31
and the scores below 2^9, so that sums in fp64 are exact in any order."""

import numpy as np
import pytest
import torch

from cache_helpers import PAGE, dev, page_table, status
from helpers import lib
from oracle.cache_oracle import route_pages_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return lib()


@pytest.mark.parametrize("n_pages,budget", [(24, 9), (200, 31), (700, 300), (2500, 40)])
@pytest.mark.parametrize("H,Hkv,D", [(4, 2, 64), (16, 1, 64), (8, 2, 128)])
def test_scores_that_only_fp64_tells_apart(sa, H, Hkv, D, n_pages, budget):
    rng = np.random.default_rng(n_pages + H)
    G, small = H // Hkv, 5
    q = rng.uniform(0.5, 1.5, (1, 1, H, D)) * rng.choice([-1, 1], (1, 1, H, D))
    q[..., small] = 1.0
    q = torch.tensor(q).to(torch.bfloat16)
    # one head of each group well above the others, so that it alone ranks the pages
    base = np.empty((Hkv, D), dtype=np.float32)
    for g in range(Hkv):
        base[g] = rng.integers(1 << 22, 3 << 22, D) * 2.0 ** -23 * np.sign(q[0, 0, g * G].float().numpy())
    step = 2.0 ** -44
    assert np.all(np.abs(q[0, 0].double().numpy()) >= 0.5)           # multiples of 2^-8
    ksum = np.broadcast_to(base, (n_pages, Hkv, D)).copy()
    # up to 256 steps above 2^16 of them: exact in fp32
    steps = rng.integers(0, 256, (n_pages, Hkv))
    ksum[:, :, small] = ((2.0 ** 16 + steps) * step).astype(np.float32)
    assert np.array_equal(ksum[:, :, small].astype(np.float64), (2.0 ** 16 + steps) * step)
    table = page_table([PAGE * n_pages], n_pages, n_pages, torch.Generator().manual_seed(1))
    lens, st = [PAGE * n_pages], status()
    rp, ci = sa.sa_route_pages(q.cuda(), torch.from_numpy(ksum).cuda(), dev(table), dev(lens), 64,
                               budget, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    want = route_pages_ref(q[:, 0].double().numpy(), ksum, table, lens, 64, budget)
    rp, ci = rp.cpu().numpy(), ci.cpu().numpy()
    for r, pages in enumerate(want):
        assert ci[rp[r]:rp[r + 1]].tolist() == pages, r
