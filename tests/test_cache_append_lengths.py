"""The lengths that sa_cache_append leaves count the tokens that it stored: what the next
sa_attn_decode attends was written."""

import numpy as np
import pytest
import torch

from cache_helpers import dev
from helpers import lib
from oracle.cache_oracle import places
from test_cache_append import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return lib()


@pytest.mark.parametrize("S", [1, 2, 130])
def test_lengths_end_where_the_rotation_tables_do(sa, S):
    """Sequences that end before, at and behind the tables' last row, and one with no room."""
    lens, rows = [0, 99, 100, 150, 40], 100
    c = Case(5, S, 2, 1, 64, "bf16", lens, rope_rows=rows, seed=S)
    place = [p for p in places(c.lens, None, S, c.max_pages) if p[2] < rows]
    c.run(sa).check(status=sa.SA_DEV_CAPACITY, place=place)
    assert c.lens_out.tolist() == [max(n, min(n + S, rows)) for n in lens]
    # a second call behind the first one stores nothing and leaves the lengths
    if S == 130:
        d = torch.zeros_like(c.lens_out)
        before = c.kbuf.clone()
        sa.sa_cache_append(c.k.cuda(), c.v.cuda(), c.kc, c.vc, dev(c.table), c.lens_out, lens_out=d,
                           cos=c.cos.cuda(), sin=c.sin.cuda())
        torch.cuda.synchronize()
        assert d.tolist() == c.lens_out.tolist() and torch.equal(before, c.kbuf)


def test_an_attention_over_the_new_lengths_meets_no_unwritten_slot(sa):
    c = Case(2, 130, 2, 1, 64, "bf16", [0, 90], rope_rows=100, seed=4)
    c.kc.fill_(float("nan"))
    c.vc.fill_(float("nan"))
    c.kc[int(c.table[1, 0])] = 0.0           # what was cached before
    c.vc[int(c.table[1, 0])] = 0.0
    c.kc[int(c.table[1, 1])][:, :26] = 0.0
    c.vc[int(c.table[1, 1])][:, :26] = 0.0
    c.run(sa)
    o, lse = sa.sa_attn_decode(c.q_out[:, :1].contiguous(), c.kc, c.vc, dev(c.table), c.lens_out)
    torch.cuda.synchronize()
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()


def test_a_page_that_is_not_there_keeps_its_place(sa):
    """Tokens behind a bad page are stored at their positions, so the length counts its own
    too; the attention leaves the page out as the append did."""
    c = Case(1, 130, 2, 1, 64, "bf16", [0], seed=5)
    c.table[0, 1] = -1
    c.kc.fill_(float("nan"))
    c.vc.fill_(float("nan"))
    place = [(b, s, t) for b, s, t in places(c.lens, None, c.S, c.max_pages) if t // 64 != 1]
    c.run(sa).check(status=sa.SA_DEV_BAD_CACHE, place=place)
    assert c.lens_out.tolist() == [130]
    o, lse = sa.sa_attn_decode(c.q_out[:, -1:].contiguous(), c.kc, c.vc, dev(c.table), c.lens_out)
    torch.cuda.synchronize()
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    assert np.isfinite(c.ksum_d.cpu().numpy()).all()
