"""sa_cache_accept and sa_cache_copy against their definitions: bytes move as they are, a
page's sum of at most 64 stored keys in fp32 is off by at most 65 roundings, each 2^-24 of
the sum of the magnitudes."""

import numpy as np
import pytest
import torch

from cache_helpers import PAGE, dev, new_cache, page_table, raw, status, values
from helpers import lib
from oracle.tree_oracle import accept_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return lib()


def some_path(rng, m, S):
    return sorted(rng.choice(S, size=m, replace=False).tolist()) + [-9] * (S - m)


class Case:
    def __init__(self, lens, S, Hkv, D, fmt, path_lens, layout="page_head", sums=True, seed=0,
                 max_pages=None, paths=None):
        gen, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
        after = [max(n, 0) + S for n in lens]
        self.max_pages = max_pages or max((n + PAGE - 1) // PAGE for n in after)
        self.lens, self.S, self.path_lens = lens, S, path_lens
        self.n_pages = sum(min((n + PAGE - 1) // PAGE, self.max_pages) for n in after) + 3
        self.table = page_table(after, self.max_pages, self.n_pages, gen)
        self.path = np.array(paths or [some_path(rng, min(m, S), S) for m in path_lens],
                             dtype=np.int32)
        fill = 1.0 if fmt == "bf16" else 40.0
        self.kc, self.kbuf = new_cache(self.n_pages, Hkv, D, fmt, layout, fill, gen)
        self.vc, self.vbuf = new_cache(self.n_pages, Hkv, D, fmt, layout, fill, gen)
        self.ks = 0.01 + 0.03 * torch.rand(Hkv, generator=gen) if fmt == "fp8" else None
        self.sum = torch.randn((self.n_pages, Hkv, D), generator=gen).cuda() if sums else None

    def expected(self):
        """Codes, as bits; sums from the values."""
        bits = [np.array(raw(t)) for t in (self.kc, self.vc)]
        k = values(self.kc)
        sums = None if self.sum is None else self.sum.cpu().double().numpy()
        scale = None if self.ks is None else self.ks.double().numpy()
        ends = accept_ref(k, k.copy(), sums, self.table, self.lens, self.path, self.path_lens, scale)
        mag = np.abs(k).sum(axis=2) * (1 if scale is None else scale[None, :, None])
        accept_ref(bits[0], bits[1], None, self.table, self.lens, self.path, self.path_lens)
        return bits, sums, mag, ends

    def run(self, sa, **kw):
        self.st = status()
        out = torch.full((len(self.lens),), -5, dtype=torch.int32, device="cuda")
        args = dict(k_sum=self.sum, k_scale=None if self.ks is None else self.ks.cuda(),
                    lens_out=out, dev_status=self.st)
        args.update(kw)
        sa.sa_cache_accept(self.kc, self.vc, dev(self.table), dev(self.lens), dev(self.path),
                           dev(self.path_lens), **args)
        torch.cuda.synchronize()
        return out

    def check(self, sa, **kw):
        bits, sums, mag, ends = self.expected()
        out = self.run(sa, **kw)
        assert np.array_equal(raw(self.kc), bits[0]) and np.array_equal(raw(self.vc), bits[1])
        assert out.tolist() == ends
        if sums is not None:
            got = self.sum.cpu().double().numpy()
            same = (self.sum_before == sums)
            assert np.array_equal(got[same], sums[same])          # pages not touched: bit for bit
            assert np.all(np.abs(got - sums) <= 65 * 2.0 ** -24 * mag + 1e-300)

    @property
    def sum_before(self):
        return self._before


def checked(sa, c, **kw):
    c._before = None if c.sum is None else c.sum.cpu().double().numpy()
    c.check(sa, **kw)
    return c


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S", [1, 2, 7, 16, 33, 64])
def test_accept_matches_the_definition(sa, S, D, fmt):
    lens = [0, 1, 62, 63, 64, 65, 100, 127, 128, 300]
    m = [(3 * i + S) % (S + 1) for i in range(10)]
    c = checked(sa, Case(lens, S, 3, D, fmt, m, seed=S + D))
    assert int(c.st.item()) == 0


@pytest.mark.parametrize("layout", ["page_token", "gapped"])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_layouts(sa, layout, fmt):
    c = Case([61, 200, 0], 9, 2, 64, fmt, [4, 9, 2], layout=layout, seed=2)
    before = raw(c.kbuf).copy(), raw(c.vbuf).copy()
    inside = torch.zeros_like(c.kbuf, dtype=torch.bool)
    view = {"page_token": lambda t: t.permute(0, 2, 1, 3),
            "gapped": lambda t: t[:c.n_pages, 1:3, :PAGE, :64]}[layout](inside)
    view.fill_(True)
    checked(sa, c)
    outside = ~inside.cpu().numpy()
    for t, b in ((c.kbuf, before[0]), (c.vbuf, before[1])):
        x = raw(t).reshape(outside.shape + (-1,)) if t.element_size() > 1 else raw(t).reshape(outside.shape)
        assert np.array_equal(x[outside], b.reshape(x.shape)[outside])


def test_nothing_accepted_takes_all_back(sa):
    """The sums are those of the keys before, so that the router ranks as before."""
    c = checked(sa, Case([100, 64, 0], 8, 2, 64, "bf16", [0, 0, 0], seed=3))
    k = values(c.kc)
    page = c.table[0, 1]
    exact = k[page, :, :36].sum(axis=1)
    assert np.allclose(c.sum.cpu().numpy()[page], exact, rtol=0, atol=37 * 2.0 ** -24 * 64 * 5)


def test_without_sums_and_lengths(sa):
    checked(sa, Case([100, 60], 8, 2, 128, "fp8", [3, 8], sums=False, seed=4))
    c = Case([100, 60], 8, 2, 128, "bf16", [3, 8], seed=4)
    bits, _, _, _ = c.expected()
    c.run(sa, lens_out=None)
    assert np.array_equal(raw(c.kc), bits[0])


def test_bad_paths_count_as_far_as_they_ascend(sa):
    paths = [[0, 2, 2, 3], [1, 0, 2, 3], [-1, 1, 2, 3], [0, 1, 64, 65], [0, 3, 5, 9], [0, 1, 2, 3]]
    c = checked(sa, Case([60] * 6, 4, 2, 64, "bf16", [4, 4, 4, 4, 4, 9], paths=paths, max_pages=2,
                         seed=5))
    # the fifth path leads beyond its sequence's last page, which is a bad page
    assert int(c.st.item()) == sa.SA_DEV_BAD_TREE | sa.SA_DEV_BAD_CACHE
    # behind the page table
    c = checked(sa, Case([124], 4, 2, 64, "bf16", [4], paths=[[0, 2, 3, 4]], max_pages=2, seed=5))
    assert int(c.st.item()) == sa.SA_DEV_BAD_TREE


def test_bad_pages_and_lengths(sa):
    c = Case([60, 61], 8, 2, 64, "bf16", [5, 5], seed=6)
    c.table[0, 1] = c.n_pages
    c = checked(sa, c)
    assert int(c.st.item()) == sa.SA_DEV_BAD_CACHE
    c = Case([10, 61], 8, 2, 64, "bf16", [5, 5], seed=6)
    c.lens = [-3, 61]
    c = checked(sa, c)
    assert int(c.st.item()) == sa.SA_DEV_BAD_CACHE


def test_accept_captured_and_refused(sa):
    c = Case([60, 100], 8, 2, 64, "bf16", [3, 2], seed=7)
    bits, _, _, ends = c.expected()
    t, n, path, m = dev(c.table), dev(c.lens), dev(c.path), dev(c.path_lens)
    m.zero_()
    out = torch.zeros_like(n)
    call = lambda **kw: sa.sa_cache_accept(c.kc, c.vc, t, n, path, m, k_sum=c.sum, **{"lens_out": out, **kw})
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    torch.cuda.synchronize()
    m.copy_(dev(c.path_lens))
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(raw(c.kc), bits[0]) and np.array_equal(raw(c.vc), bits[1])
    assert out.tolist() == ends
    for kw in (dict(lens_out=n), dict(lens_out=m)):
        with pytest.raises(sa.SaError):
            call(**kw)
    with pytest.raises(ValueError):
        sa.sa_cache_accept(c.kc, c.vc, t, n, path[:1], m)
    with pytest.raises(ValueError):
        sa.sa_cache_accept(c.kc, c.vc, t, n, path.long(), m)
    with pytest.raises(ValueError):
        sa.sa_cache_accept(c.kc, c.vc, t, n, path, None)
    with pytest.raises(sa.SaError):
        sa.sa_cache_accept(c.kc, c.vc, t, n, torch.zeros((2, 65), dtype=torch.int32, device="cuda"), m)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_accept_beyond_32_bit_offsets(sa, fmt):
    Hkv, D = 2, 128
    n_pages = (1 << 31) // (Hkv * PAGE * D) + 100
    dt = torch.bfloat16 if fmt == "bf16" else torch.uint8
    caches = [torch.zeros((n_pages, Hkv, PAGE, D), dtype=dt, device="cuda") for _ in range(2)]
    sums = torch.zeros((n_pages, Hkv, D), device="cuda")
    table = dev([[n_pages - 1, n_pages - 2]])
    for c in caches:
        c[n_pages - 2, :, 3] = 1
        c[n_pages - 1, :, 60] = 2
    sa.sa_cache_accept(caches[0], caches[1], table, dev([60]), dev([[0, 7]]), dev([2]), k_sum=sums)
    # the pair of pages moved to the front
    sa.sa_cache_copy(caches[0], caches[1], dev([[n_pages - 1, 0], [n_pages - 2, 1]]), k_sum=sums)
    torch.cuda.synchronize()
    for c in caches:
        for p in (n_pages - 1, 0):
            assert bool((c[p, :, 61] == 1).all()) and bool((c[p, :, 60] == 2).all())
        assert bool((c[1, :, 3] == 1).all())
    assert torch.equal(sums[0], sums[n_pages - 1]) and float(sums[0].abs().sum()) > 0


@pytest.mark.parametrize("layout", ["page_head", "page_token", "gapped"])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("D,Hkv", [(64, 1), (64, 5), (128, 8)])
def test_copy(sa, D, Hkv, fmt, layout):
    gen = torch.Generator().manual_seed(D + Hkv)
    n = 40
    kc, kbuf = new_cache(n, Hkv, D, fmt, layout, 1.0, gen)
    vc, vbuf = new_cache(n, Hkv, D, fmt, layout, 1.0, gen)
    sums = torch.randn((n, Hkv, D), generator=gen).cuda()
    moves = dev([[0, 39], [0, 38], [5, 3], [7, 11], [n, 2], [4, -1], [12, 13]])
    for count, done in ((None, 7), (0, 0), (3, 3), (-2, 0), (99, 7)):
        st = status()
        expect = [np.array(raw(t)) for t in (kc, vc)] + [sums.cpu().numpy().copy()]
        for a, b in moves.tolist()[:done]:
            if 0 <= a < n and 0 <= b < n:
                for x in expect:
                    x[b] = x[a]
        sa.sa_cache_copy(kc, vc, moves, None if count is None else dev([count]), k_sum=sums,
                         dev_status=st)
        torch.cuda.synchronize()
        assert np.array_equal(raw(kc), expect[0]) and np.array_equal(raw(vc), expect[1])
        assert np.array_equal(sums.cpu().numpy(), expect[2])
        assert int(st.item()) == (sa.SA_DEV_BAD_CACHE if done > 4 else 0)
    for bad in (moves[:, :1], moves.long(), moves.cpu(), moves.t()):
        with pytest.raises(ValueError):
            sa.sa_cache_copy(kc, vc, bad)
    with pytest.raises(sa.SaError):
        sa.sa_cache_copy(kc, vc, moves[:0])
