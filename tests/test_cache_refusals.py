"""Refusals of the paged-cache calls on the host, without a GPU: outputs that overlap
inputs in part, and arguments of the wrong kind."""

import ctypes

import pytest
import torch

from helpers import lib
from test_cache_host import INVALID, append, params


@pytest.fixture(scope="module")
def sa():
    return lib()


def test_lengths_out_overlap_no_lengths_in(sa):
    """B = 5 lengths: any shift of less than five entries overlaps."""
    p = params(sa, B=5)
    at = 1 << 20
    for shift in (-16, -4, 0, 4, 16):
        out = ctypes.c_void_p(at + shift)
        assert append(sa, p, lens=ctypes.c_void_p(at), lens_out=out) == INVALID, shift
        assert append(sa, p, lens=ctypes.c_void_p(2 * at), new=ctypes.c_void_p(at),
                      lens_out=out) == INVALID, shift


def test_arguments_of_the_wrong_kind(sa):
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i, n, cache = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32), z(3, 2, 64, 64)
    for kw in (dict(k_cache=cache), dict(k_cache=cache, v_cache=z(3, 2, 64)),
               dict(k_cache=z(3, 2, 64), v_cache=z(3, 2, 64)), dict(k_sum=cache)):
        with pytest.raises(ValueError):
            sa.make_cache_params(i, q=z(1, 1, 4, 64), **kw)
    with pytest.raises(ValueError):
        sa.make_cache_params(None, k_cache=cache, v_cache=cache)
    for q in (None, 1.0, [1]):
        with pytest.raises(ValueError):
            sa.sa_attn_decode(q, cache, cache, i, n)
        with pytest.raises(ValueError):
            sa.sa_route_pages(q, torch.zeros(3, 2, 64), i, n, 0, 4)
        with pytest.raises(ValueError):
            sa.sa_cache_append(q, z(1, 1, 2, 64), cache, cache, i, n)


@pytest.mark.gpu
def test_queries_of_too_few_dimensions(sa):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    i, n = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((1, 2), (1,)))
    for q in (z(64), z(4, 64), z(1, 4, 64), z(1, 1, 4, 64, 1)):
        with pytest.raises(ValueError):
            sa.sa_attn_decode(q, z(3, 2, 64, 64), z(3, 2, 64, 64), i, n)
        with pytest.raises(ValueError):
            sa.sa_route_pages(q, torch.zeros(3, 2, 64, device="cuda"), i, n, 0, 4)
        with pytest.raises(ValueError):
            sa.sa_cache_append(q, q, z(3, 2, 64, 64), z(3, 2, 64, 64), i, n)
    for pages in (None, i[0]):
        with pytest.raises(ValueError):
            sa.sa_attn_decode(z(1, 1, 4, 64), z(3, 2, 64, 64), z(3, 2, 64, 64), pages, n)
    with pytest.raises(ValueError):
        sa.sa_attn_decode(z(1, 1, 4, 64), z(3, 2, 64, 64), None, i, n)
    with pytest.raises(ValueError):
        sa.sa_attn_decode(z(1, 1, 4, 64), None, z(3, 2, 64, 64), i, n)
    torch.cuda.synchronize()
