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
