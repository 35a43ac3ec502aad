"""Forked, resized and compacted page tables against their definitions: whole numbers,
which have to be equal."""

import numpy as np
import pytest
import torch

from cache_helpers import PAGE, dev, status
from helpers import lib
from oracle.tree_oracle import compact_ref, fork_ref, resize_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return lib()


class Pool:
    """A consistent state: sequences that share full pages, pages held elsewhere, free ones."""

    def __init__(self, B, max_pages, seed=0, free=20, share=True, held=3, ahead=True):
        rng = np.random.default_rng(seed)
        self.lens = rng.integers(0, PAGE * max_pages + 1, B)
        self.lens[rng.random(B) < 0.15] = 0
        self.lens[rng.random(B) < 0.15] //= PAGE
        self.lens[rng.random(B) < 0.2] //= PAGE
        self.n_pages = B * max_pages + free + held
        ids = rng.permutation(self.n_pages).tolist()
        self.table = np.full((B, max_pages), -1, dtype=np.int32)
        self.refs = np.zeros(self.n_pages, dtype=np.int32)
        for b in range(B):
            whole, need = self.lens[b] // PAGE, -(-self.lens[b] // PAGE)
            from_other = 0
            if share and b and rng.random() < 0.5:
                c = int(rng.integers(0, b))
                from_other = int(rng.integers(0, min(whole, self.lens[c] // PAGE) + 1))
                self.table[b, :from_other] = self.table[c, :from_other]
            if ahead and rng.random() < 0.3:           # pages taken ahead
                need = min(max_pages, need + int(rng.integers(0, 3)))
            for j in range(from_other, need):
                self.table[b, j] = ids.pop()
        for p in self.table[self.table >= 0]:
            self.refs[p] += 1
        for _ in range(held):
            self.refs[ids.pop()] += 1
        self.rng = rng


def run_fork(sa, pool, src, in_place=False, **kw):
    st = status()
    refs = dev(pool.refs)
    out = sa.sa_pages_fork(dev(pool.table), dev(pool.lens), refs, dev(src), dev_status=st,
                           refs_out=refs if in_place else None, **kw)
    torch.cuda.synchronize()
    return out, int(st.item())


def check_fork(sa, pool, src, **kw):
    (table, lens, refs, moves, n), st = run_fork(sa, pool, src, **kw)
    et, el, er, em, short = fork_ref(pool.table, pool.lens, pool.refs, src)
    n = int(n.item())
    assert n == len(em) and moves[:n].tolist() == [list(m) for m in em]
    assert np.array_equal(table.cpu().numpy(), et.reshape(table.shape)) and lens.tolist() == el
    assert np.array_equal(refs.cpu().numpy(), er)
    assert bool(st & sa.SA_DEV_CAPACITY) == short
    return st


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,N,max_pages", [(1, 1, 1), (1, 5, 3), (4, 4, 7), (7, 3, 33), (40, 64, 12),
                                           (300, 300, 20), (3, 2000, 2), (2000, 9, 5)])
def test_fork(sa, B, N, max_pages, in_place):
    pool = Pool(B, max_pages, seed=B + N, free=N + 5)
    src = (B * pool.rng.random(N) ** 2).astype(np.int32)
    src[pool.rng.random(N) < 0.1] = -1
    assert check_fork(sa, pool, src, in_place=in_place) == 0


def test_fork_to_itself_and_to_nothing(sa):
    pool = Pool(20, 9, seed=4)
    assert check_fork(sa, pool, np.arange(20, dtype=np.int32)) == 0
    assert check_fork(sa, pool, np.arange(20, dtype=np.int32)[::-1].copy()) == 0
    assert check_fork(sa, pool, np.full(20, -1, dtype=np.int32)) == 0
    assert check_fork(sa, pool, np.zeros(20, dtype=np.int32)) == 0


def test_fork_without_enough_pages(sa):
    pool = Pool(6, 5, seed=1, free=0, held=0, share=False, ahead=False)
    pool.lens[:] = 100
    pool.table[:, 2:] = -1
    pool.refs[:] = 1
    pool.refs[pool.table[:, :2].max():] = 1
    free = sorted(set(range(pool.n_pages)) - set(pool.table[pool.table >= 0].tolist()))
    pool.refs[free[:2]] = 0
    for b in range(6):
        for j in range(2):
            if pool.table[b, j] < 0:
                pool.table[b, j] = free[-1 - 2 * b - j]
    assert check_fork(sa, pool, np.array([0, 0, 1, 1, 1, 2], dtype=np.int32)) == sa.SA_DEV_CAPACITY


def test_fork_of_bad_input(sa):
    pool = Pool(6, 4, seed=2)
    assert check_fork(sa, pool, np.array([0, 6, -2, 1, 99, 0], dtype=np.int32)) == sa.SA_DEV_BAD_TREE
    pool.table[3, 0] = pool.n_pages + 3
    pool.table[4, 1] = -8
    pool.lens[5] = 9999
    pool.lens[2] = -1
    st = check_fork(sa, pool, np.array([0, 3, 4, 4, 5, 2, 2, 3], dtype=np.int32))
    assert st & sa.SA_DEV_BAD_CACHE


@pytest.mark.parametrize("B,max_pages", [(1, 1), (3, 40), (50, 7), (700, 5), (4000, 3)])
def test_resize(sa, B, max_pages):
    for seed in range(3):
        pool = Pool(B, max_pages, seed=seed + B, free=B * 2 + 5)
        for more, by_sequence in ((0, False), (1, False), (70, False), (-64, False), (5, True)):
            want = pool.lens + more
            kw = {}
            if by_sequence:
                m = pool.rng.integers(-100, 150, B)
                want, kw = pool.lens + m, dict(more_lens=dev(m))
            st, table, refs = status(), dev(pool.table), dev(pool.refs)
            sa.sa_pages_resize(table, refs, dev(pool.lens), more, dev_status=st, **kw)
            torch.cuda.synchronize()
            et, er, short = resize_ref(pool.table, pool.refs, want)
            assert np.array_equal(table.cpu().numpy(), et) and np.array_equal(refs.cpu().numpy(), er)
            st = int(st.item())
            assert bool(st & sa.SA_DEV_CAPACITY) == bool(short)
            assert bool(st & sa.SA_DEV_BAD_CACHE) == bool((want < 0).any())


def test_resize_takes_and_gives_in_order(sa):
    """Pages given back in a call are not taken in it; too few pages leave the last places empty."""
    table, refs = dev([[4, 2, -1], [-1, -1, -1], [0, 5, 6]]), dev([1, 0, 1, 0, 1, 1, 1])
    st = status()
    sa.sa_pages_resize(table, refs, dev([130, 64, 64]), dev_status=st)
    assert table.tolist() == [[4, 2, 1], [3, -1, -1], [0, -1, -1]]
    assert refs.tolist() == [1, 1, 1, 1, 1, 0, 0] and int(st.item()) == 0
    sa.sa_pages_resize(table, refs, dev([192, 192, 192]), dev_status=st)
    assert table.tolist() == [[4, 2, 1], [3, 5, 6], [0, -1, -1]]
    assert int(st.item()) == sa.SA_DEV_CAPACITY and refs.tolist() == [1] * 7
    # a page that others hold as well only loses one of its places
    refs[5] = 2
    sa.sa_pages_resize(table, refs, dev([0, 64, 0]))
    assert table.tolist() == [[-1] * 3, [3, -1, -1], [-1] * 3] and refs.tolist() == [0, 0, 0, 1, 0, 1, 0]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,max_pages,free", [(1, 1, 0), (1, 1, 5), (5, 9, 0), (5, 9, 60), (40, 17, 300),
                                              (300, 30, 2000), (20, 3, 100000)])
def test_compact(sa, B, max_pages, free, in_place):
    pool = Pool(B, max_pages, seed=B + free, free=free)
    st, table, refs = status(), dev(pool.table), dev(pool.refs)
    kw = dict(table_out=table, refs_out=refs) if in_place else {}
    t, r, moves, n, used = sa.sa_pages_compact(table, refs, dev_status=st, **kw)
    torch.cuda.synchronize()
    et, er, em, eu = compact_ref(pool.table, pool.refs)
    assert int(used.item()) == eu and int(n.item()) == len(em) and int(st.item()) == 0
    assert moves[:len(em)].tolist() == [list(m) for m in em]
    assert np.array_equal(t.cpu().numpy(), et) and np.array_equal(r.cpu().numpy(), er)


def test_compact_without_a_table_and_at_the_ends(sa):
    for refs in ([0] * 70, [1] * 70, [0] * 69 + [2], [3] + [0] * 69, [0, 1] * 35, [1, 0] * 35, [5], [0]):
        t, r, moves, n, used = sa.sa_pages_compact(None, dev(refs))
        _, er, em, eu = compact_ref(np.zeros((0, 1)), refs)
        assert t is None and int(used.item()) == eu and int(n.item()) == len(em)
        assert moves[:len(em)].tolist() == [list(m) for m in em] and r.tolist() == er.tolist()


def test_strided_tables_and_dirty_workspaces(sa):
    pool = Pool(12, 6, seed=9, free=40)
    src = np.array([3, 3, 1, -1, 0, 11, 3], dtype=np.int32)
    wide = torch.full((12, 11), 77, dtype=torch.int32, device="cuda")
    table = wide[:, 2:8]
    table.copy_(dev(pool.table))
    out = torch.full((7, 9), 55, dtype=torch.int32, device="cuda")
    ws = torch.full((sa.sa_pages_workspace_bytes(pool.n_pages, 12),), 0xA5, dtype=torch.uint8, device="cuda")
    refs = dev(pool.refs)
    t, lens, r, moves, n = sa.sa_pages_fork(table, dev(pool.lens), refs, dev(src), table_out=out[:, 1:7],
                                            workspace=ws)
    et, el, er, em, _ = fork_ref(pool.table, pool.lens, pool.refs, src)
    assert np.array_equal(t.cpu().numpy(), et) and lens.tolist() == el and r.tolist() == er.tolist()
    assert bool((out[:, :1] == 55).all()) and bool((out[:, 7:] == 55).all())
    ws.fill_(0x5A)
    t2, r2, moves, n, used = sa.sa_pages_compact(table, refs, table_out=table, refs_out=refs, workspace=ws)
    et, er, em, eu = compact_ref(pool.table, pool.refs)
    assert np.array_equal(table.cpu().numpy(), et) and refs.tolist() == er.tolist()
    ws.fill_(0xFF)
    sa.sa_pages_resize(table, refs, dev(pool.lens), 64, workspace=ws)
    et, er, _ = resize_ref(et, er, pool.lens + 64)
    assert np.array_equal(table.cpu().numpy(), et) and refs.tolist() == er.tolist()
    assert bool((wide[:, :2] == 77).all()) and bool((wide[:, 8:] == 77).all())


def test_captured_and_replayed(sa):
    """A step of beams as a graph: fork, room for a token, the copies, all on fixed buffers."""
    pool = Pool(10, 5, seed=3, free=60)
    N = 10
    table, lens, refs = dev(pool.table), dev(pool.lens), dev(pool.refs)
    src = torch.zeros(N, dtype=torch.int32, device="cuda")
    kc = torch.arange(pool.n_pages, dtype=torch.bfloat16, device="cuda")[:, None, None, None]
    kc = kc.expand(-1, 2, PAGE, 64).contiguous()
    vc = kc.clone()
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    buf = dict(table_out=z(N, 5), lens_out=z(N), refs_out=torch.zeros_like(refs), moves=z(N, 2), n_moves=z(1),
               workspace=torch.empty(sa.sa_pages_workspace_bytes(pool.n_pages, N), dtype=torch.uint8, device="cuda"))

    def step():
        sa.sa_pages_fork(table, lens, refs, src, **buf)
        sa.sa_pages_resize(buf["table_out"], buf["refs_out"], buf["lens_out"], 1, workspace=buf["workspace"])
        sa.sa_cache_copy(kc, vc, buf["moves"], buf["n_moves"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    for seed in range(4):
        pages = torch.arange(pool.n_pages, dtype=torch.bfloat16, device="cuda")[:, None, None, None]
        kc.copy_(pages.expand_as(kc))
        vc.copy_(kc)
        s = np.random.default_rng(seed).integers(-1, 10, N).astype(np.int32)
        src.copy_(dev(s))
        graph.replay()
        torch.cuda.synchronize()
        t, el, r, em, _ = fork_ref(pool.table, pool.lens, pool.refs, s)
        t, r, _ = resize_ref(t, r, np.array(el) + 1)
        assert np.array_equal(buf["table_out"].cpu().numpy(), t) and buf["lens_out"].tolist() == el
        assert buf["refs_out"].tolist() == r.tolist()
        for a, b in em:
            assert bool((kc[b] == kc[a, 0, 0, 0]).all()) and bool((vc[b] == kc[a, 0, 0, 0]).all())


def test_calls_behind_each_other_and_on_two_streams(sa):
    """Each call sees what the ones before it on its stream have written, without a wait of
    the host, while another stream does the same with another pool."""
    pools = [Pool(24, 6, seed=40 + i, free=80) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in pools]
    rng = np.random.default_rng(1)
    srcs = [[rng.integers(-1, 24, 24).astype(np.int32) for _ in range(6)] for _ in pools]
    state = [[dev(p.table), dev(p.lens), dev(p.refs)] for p in pools]
    src = [[dev(s) for s in x] for x in srcs]
    kc = [torch.zeros((p.n_pages, 1, PAGE, 64), dtype=torch.bfloat16, device="cuda") for p in pools]
    big = torch.ones(1 << 26, device="cuda")
    torch.cuda.synchronize()
    for step in range(6):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                table, lens, refs = state[i]
                late = (big * 0).sum().int() + src[i][step]        # ready only when that is done
                table, lens, refs, moves, n = sa.sa_pages_fork(table, lens, refs, late)
                sa.sa_pages_resize(table, refs, lens, 1)
                sa.sa_cache_copy(kc[i], kc[i].clone(), moves, n)
                lens = lens.clamp(max=6 * PAGE - 1) + 1
                sa.sa_pages_resize(table, refs, lens)
                table, refs, moves, n, used = sa.sa_pages_compact(table, refs)
                state[i] = [table, lens, refs]
    torch.cuda.synchronize()
    for p, x, (table, lens, refs) in zip(pools, srcs, state):
        t, l, r = p.table, p.lens, p.refs
        for s in x:
            t, l, r, _, _ = fork_ref(t, l, r, s)
            l = np.array(l)
            t, r, _ = resize_ref(t, r, l + 1)
            l = np.minimum(l, 6 * PAGE - 1) + 1
            t, r, _ = resize_ref(t, r, l)
            t, r, *_ = compact_ref(t, r)
        assert np.array_equal(table.cpu().numpy(), t) and lens.tolist() == l.tolist()
        assert refs.tolist() == list(r)


def test_refusals(sa):
    pool = Pool(5, 4, seed=1)
    t, n, r, src = dev(pool.table), dev(pool.lens), dev(pool.refs), dev([0, 1, 2])
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    fork = lambda **kw: sa.sa_pages_fork(**{**dict(page_table=t, seq_lens=n, refs=r, src=src), **kw})
    fork()
    for kw in (dict(page_table=t.long()), dict(page_table=t.t()), dict(seq_lens=n[:3]), dict(refs=r.float()),
               dict(src=src.long()), dict(src=src[None]), dict(table_out=z(3, 3)), dict(table_out=z(4, 4)),
               dict(lens_out=z(2)), dict(refs_out=z(3)), dict(moves=z(2, 2)), dict(moves=z(3, 3)),
               dict(n_moves=z(2)), dict(src=src.cpu()), dict(workspace=z(64)[::2])):
        with pytest.raises(ValueError):
            fork(**kw)
    for kw in (dict(table_out=t[:3]), dict(lens_out=n[1:4]), dict(workspace=z(8)),
               dict(page_table=t[:0], seq_lens=n[:0]), dict(src=src[:0])):
        with pytest.raises((ValueError, sa.SaError)):
            fork(**kw)
    big = torch.zeros(2 * pool.n_pages, dtype=torch.int32, device="cuda")
    with pytest.raises(sa.SaError):
        fork(refs=big[:pool.n_pages], refs_out=big[1:pool.n_pages + 1])
    for kw in (dict(table_out=z(5, 3)), dict(refs_out=z(3)), dict(moves=z(2, 2)), dict(n_used=z(2)),
               dict(n_moves=z(3))):
        with pytest.raises(ValueError):
            sa.sa_pages_compact(t, r, **kw)
    with pytest.raises(ValueError):
        sa.sa_pages_compact(None, r, table_out=z(5, 4))
    wide = torch.zeros((6, 4), dtype=torch.int32, device="cuda")
    with pytest.raises(sa.SaError):
        sa.sa_pages_compact(wide[:5], r, table_out=wide[1:])
    for bad in (dict(page_table=t.float()), dict(refs=r.long()), dict(seq_lens=n[:2]), dict(more_lens=z(2)),
                dict(more=1.5), dict(more=1 << 40)):
        with pytest.raises(ValueError):
            sa.sa_pages_resize(**{**dict(page_table=t.clone(), refs=r.clone(), seq_lens=n), **bad})
    torch.cuda.synchronize()
