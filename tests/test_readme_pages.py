"""The README's lines on the pool's pages, run as they stand: afterwards each sequence holds
what the one it continues held, in every layer, and the counts are those of the table."""

import os

import numpy as np
import pytest
import torch

from cache_helpers import PAGE, dev
from helpers import lib

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def block_with(name):
    """The README's Python lines that call `name`."""
    with open(README) as f:
        blocks = [b.split("```")[0] for b in f.read().split("```python\n")[1:]]
    found = [b for b in blocks if name + "(" in b]
    assert len(found) == 1
    return found[0]


def held(cache, table, lens):
    """What each sequence holds of a cache [n_pages, H_kv, 64, D], tokens in order."""
    out = []
    for b, n in enumerate(lens):
        pages = [cache[int(table[b, j])] for j in range(-(-n // PAGE))]
        out.append(torch.cat(pages, 1)[:, :n] if pages else None)
    return out


def test_pages():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sa = lib()
    gen = torch.Generator().manual_seed(1)
    n_pages, Hkv, D, B, most = 64, 2, 64, 4, 5
    lens = [130, 64, 0, 200]
    table = np.full((B, most), -1, dtype=np.int32)
    ids = (60 - 4 * np.arange(15)).tolist()            # far apart, so that most of them move
    for b, n in enumerate(lens):
        for j in range(-(-n // PAGE)):
            table[b, j] = ids.pop(0)
    refs = np.zeros(n_pages, dtype=np.int32)
    refs[table[table >= 0]] = 1
    layers = [tuple(torch.randn((n_pages, Hkv, PAGE, D), generator=gen).to(torch.bfloat16).cuda()
                    for _ in range(2)) + (torch.randn((n_pages, Hkv, D), generator=gen).cuda(),)
              for _ in range(2)]
    was = [(held(k, table, lens), held(v, table, lens), s.clone()) for k, v, s in layers]
    src = [3, 0, 3, 1, 0]
    names = dict(sa=sa, table=dev(table), lens=dev(lens), refs=dev(refs), src=dev(src), layers=layers)
    exec(block_with("sa_pages_fork"), names)
    torch.cuda.synchronize()
    new, n = names["table"].cpu().numpy(), names["lens"].tolist()
    assert n == [lens[i] for i in src]
    assert np.array_equal(np.bincount(new[new >= 0], minlength=n_pages), names["refs"].cpu().numpy())
    used = int(names["used"].item())
    assert int(new.max()) < used == int((names["refs"] > 0).sum())
    for (k, v, s), (k0, v0, s0) in zip(layers, was):
        for i, (a, b) in enumerate(zip(held(k, new, n), held(v, new, n))):
            assert torch.equal(a, k0[src[i]]) and torch.equal(b, v0[src[i]])
            for j in range(-(-n[i] // PAGE)):
                assert torch.equal(s[int(new[i, j])], s0[int(table[src[i], j])])
