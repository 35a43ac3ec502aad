"""What the pages hold, behind forks, resizes and compactions that follow each other on a
stream without a wait of the host: every page of the pool, bit for bit."""

import numpy as np
import pytest
import torch

from cache_helpers import PAGE, dev
from helpers import lib
from oracle.tree_oracle import compact_ref, fork_ref, resize_ref
from test_pages import Pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return lib()


def some_cache(n_pages, Hkv, D, fmt, gen):
    """Bytes of no order (0 to 126: no NaN in e4m3), another for every page."""
    n = D * (1 if fmt == "fp8" else 2)
    x = torch.randint(0, 127, (n_pages, Hkv, PAGE, n), generator=gen, dtype=torch.uint8).cuda()
    return x.view(torch.float8_e4m3fn if fmt == "fp8" else torch.bfloat16)


def as_bytes(t):
    return t.view(torch.uint8)


@pytest.mark.parametrize("fmt,Hkv,D", [("bf16", 3, 64), ("fp8", 2, 128), ("fp8", 1, 64)])
@pytest.mark.parametrize("busy", [False, True])
def test_copies_behind_forks_and_compactions(sa, busy, fmt, Hkv, D):
    """Two pools on two streams; a third stream keeps the SMs busy, so that the CTAs of a call
    come late and one by one."""
    steps, B, most = 6, 24, 6
    pools = [Pool(B, most, seed=60 + i, free=80) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in pools]
    rng, gen = np.random.default_rng(2), torch.Generator().manual_seed(D)
    srcs = [[rng.integers(-1, B, B).astype(np.int32) for _ in range(steps)] for _ in pools]
    state = [[dev(p.table), dev(p.lens), dev(p.refs)] for p in pools]
    src = [[dev(s) for s in x] for x in srcs]
    first = [[some_cache(p.n_pages, Hkv, D, fmt, gen) for _ in range(2)] +
             [torch.rand((p.n_pages, Hkv, D), generator=gen).cuda()] for p in pools]
    now = [[t.clone() for t in x] for x in first]
    big = torch.ones(1 << 26, device="cuda")
    load = torch.ones((2048, 2048), device="cuda")
    third = torch.cuda.Stream()
    torch.cuda.synchronize()
    for step in range(steps):
        if busy:
            with torch.cuda.stream(third):
                for _ in range(20):
                    load @ load
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                table, lens, refs = state[i]
                kc, vc, ks = now[i]
                late = (big * 0).sum().int() + src[i][step]        # ready only when that is done
                table, lens, refs, moves, n = sa.sa_pages_fork(table, lens, refs, late)
                sa.sa_pages_resize(table, refs, lens, 1)
                sa.sa_cache_copy(kc, vc, moves, n, k_sum=ks)
                table, refs, moves, n, used = sa.sa_pages_compact(table, refs)
                sa.sa_cache_copy(kc, vc, moves, n, k_sum=ks)
                state[i] = [table, lens.clone(), refs]
    torch.cuda.synchronize()
    for p, x, (table, lens, refs), was, got in zip(pools, srcs, state, first, now):
        t, l, r = p.table, p.lens, p.refs
        holds = np.arange(p.n_pages)                     # the page whose contents a page has
        for s in x:
            t, l, r, m, _ = fork_ref(t, l, r, s)
            l = np.array(l)
            t, r, _ = resize_ref(t, r, l + 1)
            for a, b in m:
                holds[b] = holds[a]
            t, r, m, _ = compact_ref(t, r)
            for a, b in m:
                holds[b] = holds[a]
        assert np.array_equal(table.cpu().numpy(), t) and lens.tolist() == l.tolist()
        assert refs.tolist() == list(r)
        at = dev(holds, torch.int64)
        for a, b in zip(was, got):
            assert torch.equal(as_bytes(b), as_bytes(a)[at])


@pytest.mark.parametrize("B,max_pages,free", [(4, 3, 300), (300, 5, 9000)])
def test_the_same_beside_a_busy_stream(sa, B, max_pages, free):
    """The counts of a cluster's CTAs reach each other whenever those begin: some hundred calls
    while other kernels come and go on the SMs."""
    pool = Pool(B, max_pages, seed=B, free=free)
    src = dev((B * pool.rng.random(B) ** 2).astype(np.int32))
    table, lens, refs = dev(pool.table), dev(pool.lens), dev(pool.refs)
    load = torch.ones((1024, 1024), device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    first, differ = None, torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(300):
        with torch.cuda.stream(side):
            for _ in range(i % 4):
                load @ load
        t, l, r, moves, n = sa.sa_pages_fork(table, lens, refs, src)
        sa.sa_pages_resize(t, r, l, 64)
        c, s, m, k, used = sa.sa_pages_compact(t, r)
        out = [t, l, r, n, c, s, k, used]
        if first is None:
            first = [x.clone() for x in out]
        for a, b in zip(first, out):
            differ += (a != b).any().long()
    torch.cuda.synchronize()
    assert int(differ.item()) == 0
    et, el, er, em, _ = fork_ref(pool.table, pool.lens, pool.refs, src.cpu().numpy())
    et, er, _ = resize_ref(et, er, np.array(el) + 64)
    ct, cr, cm, cu = compact_ref(et, er)
    for got, exp in zip(first, [et, el, er, [len(em)], ct, cr, [len(cm)], [cu]]):
        assert np.array_equal(got.cpu().numpy(), np.asarray(exp))
