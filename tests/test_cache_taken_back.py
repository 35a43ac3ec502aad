"""Tokens taken back from a paged cache (a guess that was rejected): the length is set
back and the sums of the page that the sequence then ends in are put back, as sa.h says."""

import numpy as np
import pytest
import torch

from cache_helpers import PAGE, dev, raw
from helpers import lib
from test_cache_append import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return lib()


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("S", [1, 3, 70])
def test_tokens_taken_back_leave_no_trace(sa, S, fmt):
    lens = [100, 128, 63, 0, 190]             # inside pages, at an edge, at the start
    c = Case(5, S, 2, 2, 64, fmt, lens, seed=S)
    d = Case(5, S, 2, 2, 64, fmt, lens, seed=S)
    guess = torch.randn(c.k.shape, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16)
    keep = [int(c.table[b, n // PAGE]) for b, n in enumerate(lens)]
    saved = c.ksum_d[keep].clone()
    k, v = c.k, c.v
    c.k = c.v = guess
    c.run(sa)
    c.ksum_d[keep] = saved                     # taken back: lens is what it was before
    c.k, c.v = k, v
    c.run(sa)
    d.run(sa)
    assert torch.equal(c.ksum_d, d.ksum_d) and torch.equal(c.lens_out, d.lens_out)
    assert np.array_equal(raw(c.kbuf), raw(d.kbuf)) and np.array_equal(raw(c.vbuf), raw(d.vbuf))
