"""sa_route_pages where single heads of a page score no number: those are passed over."""

import numpy as np
import pytest
import torch

from helpers import lib
from test_cache_route import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return lib()


@pytest.mark.parametrize("n_pages", [30, 400])
@pytest.mark.parametrize("H,Hkv", [(4, 2), (24, 2)])
def test_a_head_without_a_number_is_passed_over(sa, H, Hkv, n_pages):
    c = Case([64 * n_pages], H, Hkv, 64, seed=n_pages)
    t, G = c.table[0], H // Hkv
    c.q[0, 0, 0, 5] = 0.0                      # 0 times infinity for the first head alone
    c.ksum[t[3], 0, 5] = float("-inf")         # the others: minus or plus infinity
    c.ksum[t[4], 0, 5] = float("inf")
    c.q[0, 0, G, 7] = float("nan")             # a head that has no number anywhere
    for budget in (3, 9, n_pages - 2):
        rp, ci = c.run(sa, 0, budget)
        c.check(rp, ci, 0, budget)
    c.q[0, 0, :, 7] = float("nan")             # none has: the first pages
    rp, ci = c.run(sa, 0, 9)
    c.check(rp, ci, 0, 9)
    assert ci[rp[0]:rp[1]].tolist() == list(range(8)) + [n_pages - 1]
    assert np.all(np.diff(rp) == 9)
