"""sa_attn_decode over a route where many query heads share a key-value head: two and four
groups of 16 rows, and several CTAs' worth of rows (more than 64 heads), with units that are
cut between runs, in rows that one warp finds and in more than that. Bounds as in
test_cache_decode.py."""

import numpy as np
import pytest
import torch

from helpers import lib
from test_cache_decode import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return lib()


def some_rows(lens, Hkv, rng, share):
    rows = []
    for n in lens:
        nb = (n + 63) // 64
        for _ in range(Hkv):
            m = int(rng.integers(0, nb + 1)) if share is None else int(nb * share)
            rows.append(sorted(rng.choice(nb, size=m, replace=False).tolist()))
    return rows


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("H,Hkv", [(8, 1), (9, 1), (16, 1), (32, 1), (56, 1), (130, 2), (129, 1)])
def test_few_long_rows_are_cut(sa, H, Hkv, fmt, D):
    lens = [64 * 330 - 5, 0, 64 * 120, 70]
    c = Case(lens, H, Hkv, D, fmt, seed=H + D)
    rows = some_rows(lens, Hkv, np.random.default_rng(H), 0.8)
    o, lse = c.run(sa, rows)
    assert int(c.st.item()) == 0
    c.check(o, lse, rows)
    again, lse2 = c.run(sa, rows)
    assert torch.equal(o, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("H,Hkv,B", [(32, 1, 45), (56, 1, 45), (130, 2, 30), (100, 1, 33)])
def test_many_rows(sa, H, Hkv, B, fmt, D):
    lens = [(173 * i) % 1500 for i in range(B)]
    lens[7] = 64 * 200 + 1
    c = Case(lens, H, Hkv, D, fmt, seed=H + D + 1)
    rows = some_rows(lens, Hkv, np.random.default_rng(H), None)
    rows[7 * Hkv] = list(range(201))
    o, lse = c.run(sa, rows)
    assert int(c.st.item()) == 0
    c.check(o, lse, rows)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("H,Hkv", [(65, 1), (130, 2), (200, 1)])
def test_more_than_64_heads_without_a_route(sa, H, Hkv, fmt, D):
    c = Case([64 * 250 + 9, 64, 0, 131], H, Hkv, D, fmt, seed=H)
    o, lse = c.run(sa)
    assert int(c.st.item()) == 0
    c.check(o, lse)
    rows = [list(range((n + 63) // 64)) for n in c.lens for _ in range(Hkv)]
    x, y = c.run(sa, rows)                     # every page listed: the same bits
    assert torch.equal(o, x) and torch.equal(lse, y)
