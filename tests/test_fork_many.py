"""Forks of many sequences, whose counts take more shared memory than a kernel has unasked."""

import ctypes
import threading

import numpy as np
import pytest
import torch

from cache_helpers import dev
from helpers import lib
from oracle.tree_oracle import fork_ref
from test_pages import Pool, check_fork

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return lib()


@pytest.mark.parametrize("B,N,max_pages", [(5120, 3, 1), (5121, 70, 1), (5121, 5121, 2), (12000, 9, 1),
                                           (16384, 1, 1), (16384, 16384, 1)])
def test_fork(sa, B, N, max_pages):
    pool = Pool(B, max_pages, seed=B + N, free=N + 5)
    src = (B * pool.rng.random(N) ** 2).astype(np.int32)
    src[pool.rng.random(N) < 0.1] = -1
    assert check_fork(sa, pool, src) == 0
    assert check_fork(sa, pool, src, in_place=True) == 0


def test_threads_with_forks_of_different_sizes(sa):
    """Two threads of the host, by the C entry point (a call of it leaves the interpreter): what
    one asks for does not take from what the other has asked for."""
    c = sa.load_library()
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    bad, outs = [], {}
    go = threading.Barrier(2)
    pools = {B: Pool(B, 1, seed=B, free=40) for B in (5200, 16384)}

    def work(B):
        pool = pools[B]
        N = 16
        st = torch.cuda.Stream()
        src = np.arange(0, 3 * N, 3, dtype=np.int32) // 2
        table, lens, refs, s = dev(pool.table), dev(pool.lens), dev(pool.refs), dev(src)
        t, l, r, m, n, status = i32(N, 1), i32(N), i32(pool.n_pages), i32(N, 2), i32(1), i32(1)
        ws = torch.empty(sa.sa_pages_workspace_bytes(pool.n_pages, B), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        p = lambda x: ctypes.c_void_p(x.data_ptr())
        args = (pool.n_pages, 1, B, N, p(table), 1, p(lens), p(refs), p(s), p(t), 1, p(l), p(r), p(m),
                p(n), p(ws), ws.numel(), p(status), ctypes.c_void_p(st.cuda_stream))
        go.wait()
        for _ in range(3000):
            code = c.sa_pages_fork(*args)
            if code:
                bad.append((B, code))
                break
        st.synchronize()
        outs[B] = (src, t, l, r, status)

    threads = [threading.Thread(target=work, args=(B,)) for B in pools]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    for B, (src, t, l, r, status) in outs.items():
        et, el, er, _, _ = fork_ref(pools[B].table, pools[B].lens, pools[B].refs, src)
        assert np.array_equal(t.cpu().numpy(), et) and l.tolist() == el
        assert np.array_equal(r.cpu().numpy(), er) and int(status.item()) == 0
