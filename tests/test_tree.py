"""sa_attn_tree against the fp64 definition.

Bounds, from the arithmetic, as those of one new token: a logit's products are exact in
fp32 and summed with an error of at most (D + 4) 2^-24 of scale sum |q k|; its scaling,
the subtraction of the maximum and the exponential add 2^-22 of the logit's and of one
part: dl. A weight is rounded to 2^-16 of itself (2^-11 over a cache in e4m3), the sums of
n weights in fp32 are off by at most n 2^-24. So
  |o - exact| <= 2^-8 |exact| + (2 dl + 2^-16 or 2^-11 + 2 n 2^-24) sum a |v|,
  |lse - exact| <= dl + n 2^-24 + 2^-22 (|lse| + 1)."""

import math

import numpy as np
import pytest
import torch

from cache_helpers import PAGE, dev, new_cache, page_table, status, values
from helpers import lib
from oracle.tree_oracle import ancestors_ref, new_tokens_ref, tree_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return lib()


def random_parents(B, S, rng, forest=0.1):
    up = np.full((B, S), -1, dtype=np.int32)
    for b in range(B):
        for s in range(1, S):
            if rng.random() >= forest:
                up[b, s] = rng.integers(0, s)
    return up


class Case:
    def __init__(self, lens, S, H, Hkv, D, fmt, new=None, parents="random", layout="page_head",
                 scale=0.0, qmag=2.0, seed=0, max_pages=None, garbage=True):
        gen, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
        self.__dict__.update(lens=lens, S=S, H=H, Hkv=Hkv, D=D, fmt=fmt, new=new, scale=scale)
        B = len(lens)
        after = [max(n, 0) + (S if new is None else min(max(new[b], 0), S)) for b, n in enumerate(lens)]
        need = [(n + PAGE - 1) // PAGE for n in after]
        self.max_pages = max_pages or max(1, max(need))
        self.n_pages = sum(min(x, self.max_pages) for x in need) + 2
        self.table = page_table(after, self.max_pages, self.n_pages, gen)
        self.parents = random_parents(B, S, rng) if isinstance(parents, str) else parents
        self.q = (qmag * torch.randn((B, S, H, D), generator=gen)).to(torch.bfloat16)
        fill = 1.0 if fmt == "bf16" else 40.0
        self.kc, _ = new_cache(self.n_pages, Hkv, D, fmt, layout, fill, gen)
        self.vc, _ = new_cache(self.n_pages, Hkv, D, fmt, layout, fill, gen)
        self.ks = self.vs = None
        if fmt == "fp8":
            self.ks = 0.01 + 0.03 * torch.rand(Hkv, generator=gen)
            self.vs = 0.01 + 0.03 * torch.rand(Hkv, generator=gen)
        if garbage:                    # what lies behind a sequence's last token has no effect
            for b, n in enumerate(after):
                if n % PAGE and 0 < n <= PAGE * self.max_pages:
                    self.put(b, n, None, float("nan"))
                    if n % PAGE < 62:
                        self.put(b, n + 1, n + 2, float("inf"))

    def put(self, b, lo, hi, x, caches=("kc", "vc")):
        """x (NaN, or inf where there is one) into the slots of tokens lo .. hi of a page."""
        page = int(self.table[b, lo // PAGE])
        hi = PAGE if hi is None else (hi - 1) % PAGE + 1
        for name in caches:
            t = getattr(self, name)
            if self.fmt == "bf16":
                t[page, :, lo % PAGE:hi] = x
            else:
                t.view(torch.uint8)[page, :, lo % PAGE:hi] = 0x7F

    def run(self, sa, rows=None, **kw):
        c = lambda t: None if t is None else t.cuda()
        self.st = status()
        shape = (len(self.lens), self.S, self.H, self.D)
        self.o0 = torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")
        self.l0 = torch.full((shape[0], self.H, self.S), 7.0, device="cuda")
        args = dict(scale=self.scale, parents=dev(self.parents), new_lens=dev(self.new),
                    k_scale=c(self.ks), v_scale=c(self.vs), dev_status=self.st, o=self.o0,
                    lse=self.l0)
        if rows is not None:
            rp = np.concatenate([[0], np.cumsum([len(r) for r in rows])])
            ci = np.concatenate([np.asarray(r, dtype=np.int64) for r in rows] + [[0]])
            args.update(row_ptr=dev(rp), col_idx=dev(ci))
        args.update(kw)
        o, lse = sa.sa_attn_tree(c(self.q), self.kc, self.vc, dev(self.table), dev(self.lens),
                                 **args)
        torch.cuda.synchronize()
        return o, lse

    def check(self, o, lse, rows=None):
        scale = self.scale or 1 / math.sqrt(self.D)
        k, v = values(self.kc, self.ks), values(self.vc, self.vs)
        q = self.q.double().numpy()
        with np.errstate(invalid="ignore"):
            eo, el, mag, written = tree_ref(q, k, v, self.table, self.lens, self.new, self.parents,
                                            scale, rows)
        knorm = np.linalg.norm(np.nan_to_num(k, posinf=0, neginf=0), axis=-1).max()
        top = scale * np.linalg.norm(q, axis=-1) * knorm                    # [B, S, H]
        n = np.array([a + m for a, m in new_tokens_ref(self.lens, self.new, self.S, self.max_pages)])
        n = n[:, None, None]
        dl = top * ((self.D + 4) * 2.0 ** -24 + 2.0 ** -22) + 2.0 ** -22
        w = 2 * dl + (2.0 ** -16 if self.fmt == "bf16" else 2.0 ** -11) + 2 * n * 2.0 ** -24
        got = o.cpu().double().numpy()
        assert np.all(got[~written] == 7.0)                  # rows without a token stay
        tol = 2.0 ** -8 * np.abs(eo) + w[..., None] * mag
        fine = np.isfinite(eo) & written[:, :, None, None]
        assert np.array_equal(np.isnan(got[written]), np.isnan(eo[written]))
        odd = np.isinf(eo)
        assert np.array_equal(got[odd], eo[odd])
        off = np.abs(np.where(fine, got, 0) - np.where(fine, eo, 0))
        tol = np.where(fine, tol, 1)
        assert np.all(off <= tol), float(np.max(off / np.maximum(tol, 1e-30)))
        if lse is not None:
            gl = lse.cpu().double().numpy().transpose(0, 2, 1)              # [B, S, H]
            el = el.transpose(0, 2, 1)
            assert np.all(gl[~written] == 7.0)
            empty = np.isneginf(el)
            assert np.array_equal(np.isneginf(gl[written]), empty[written])
            ok = written[:, :, None] & np.isfinite(el)
            tl = dl + n * 2.0 ** -24 + 2.0 ** -22 * (np.abs(np.where(ok, el, 0)) + 1)
            assert np.all(np.abs(np.where(ok, gl, 0) - np.where(ok, el, 0)) <= tl)


LENS = [[0], [1], [63], [64], [65], [129, 0, 1, 64], [777], [1500, 5, 700]]


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S", [1, 2, 3, 8, 13, 33, 64])
@pytest.mark.parametrize("lens", LENS, ids=lambda l: f"{len(l)}x{max(l)}")
def test_lengths(sa, lens, S, D, fmt):
    c = Case(lens, S, 8, 2, D, fmt, seed=len(lens) + S + D)
    o, lse = c.run(sa)
    assert int(c.st.item()) == 0
    c.check(o, lse)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S", [5, 16])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 4), (5, 1), (7, 1), (16, 2), (17, 1), (33, 1), (56, 8),
                                   (56, 1), (100, 1)])
def test_head_layouts(sa, H, Hkv, S, D, fmt):
    """From 5 to 1,600 rows on a key-value head."""
    c = Case([300, 64, 17], S, H, Hkv, D, fmt, new=[S, S - 2, 1], seed=H + S)
    o, lse = c.run(sa)
    assert int(c.st.item()) == 0
    c.check(o, lse)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("H,Hkv", [(4, 2), (48, 4)])
def test_unequal_trees_and_empty_ones(sa, H, Hkv, fmt):
    """Sequences without a new token are left alone, whatever else they are."""
    lens = [0, 1, 63, 64, 200, 127, 300, 61, 128, 5, 0]
    new = [0, 9, 1, 0, 16, 2, 15, 3, 7, 16, 4]
    c = Case(lens, 16, H, Hkv, 128, fmt, new=new, seed=3)
    o, lse = c.run(sa)
    assert int(c.st.item()) == 0
    c.check(o, lse)


@pytest.mark.parametrize("G", [2, 24])
def test_trees_of_every_form(sa, G):
    S = 64
    chain = np.arange(-1, S - 1, dtype=np.int32)
    star = np.array([-1] + [0] * (S - 1), dtype=np.int32)
    alone = np.full(S, -1, dtype=np.int32)
    binary = np.array([-1] + [(s - 1) // 2 for s in range(1, S)], dtype=np.int32)
    comb = np.array([-1] + [s - 1 if s % 2 else max(s - 2, 0) for s in range(1, S)], dtype=np.int32)
    for base in (0, 1, 40, 63, 64, 100):
        c = Case([base] * 5, S, 2 * G, 2, 64, "bf16", parents=np.stack([chain, star, alone, binary, comb]),
                 seed=base)
        o, lse = c.run(sa)
        assert int(c.st.item()) == 0
        c.check(o, lse)
    # no parents: each continues the one before it
    c.parents = np.tile(chain, (5, 1))
    with_parents, _ = c.run(sa)
    with_parents = with_parents.clone()
    c.parents = None
    assert torch.equal(c.run(sa)[0], with_parents)
    # one tree for all
    c.parents = np.tile(binary, (5, 1))
    each, _ = c.run(sa)
    each = each.clone()
    assert torch.equal(c.run(sa, parents=dev(binary))[0], each)
    shared = torch.from_numpy(binary).cuda()[None].expand(5, S)
    assert torch.equal(c.run(sa, parents=shared)[0], each)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("H,Hkv,S", [(8, 2, 1), (8, 1, 1), (12, 1, 1), (16, 2, 4), (24, 1, 2), (56, 4, 16)])
def test_long_and_short_contexts_together(sa, H, Hkv, S, fmt):
    c = Case([6000, 0, 3, 64, 1000, 130], S, H, Hkv, 128, fmt, seed=S + H)
    o, lse = c.run(sa)
    assert int(c.st.item()) == 0
    c.check(o, lse)


@pytest.mark.parametrize("H,Hkv", [(4, 4), (40, 2)])
def test_many_sequences(sa, H, Hkv):
    lens = [(53 * i) % 190 for i in range(300)]
    new = [i % 6 for i in range(300)]
    c = Case(lens, 5, H, Hkv, 64, "bf16", new=new, seed=1)
    o, lse = c.run(sa)
    assert int(c.st.item()) == 0
    c.check(o, lse)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S,G", [(16, 1), (17, 1), (5, 5), (4, 8), (11, 3), (1, 32), (3, 43), (2, 64), (64, 2)])
def test_rows_next_to_the_tiles_sizes(sa, S, G, D, fmt):
    """16 to 129 rows on a key-value head, tables small and large."""
    lens = [(71 * i) % 400 for i in range(12)]
    for max_pages in (None, 40):
        c = Case(lens, S, 3 * G, 3, D, fmt, seed=S, max_pages=max_pages)
        o, lse = c.run(sa)
        assert int(c.st.item()) == 0
        c.check(o, lse)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("layout", ["page_token", "gapped"])
@pytest.mark.parametrize("H", [6, 48])
def test_cache_layouts(sa, layout, fmt, H):
    c = Case([500, 70, 64], 7, H, 3, 128, fmt, layout=layout, seed=9)
    o, lse = c.run(sa)
    c.check(o, lse)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("H", [4, 48])
def test_peaked_softmax(sa, fmt, H):
    c = Case([700, 90], 9, H, 2, 128, fmt, qmag=40.0, seed=5)
    o, lse = c.run(sa)
    c.check(o, lse)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("H,Hkv", [(8, 2), (32, 2), (56, 1)])
def test_routed_pages(sa, H, Hkv, fmt):
    """Pages with new tokens are attended whether a row lists them or not."""
    rng = np.random.default_rng(2)
    lens, new = [3000, 64, 40, 127, 1000, 640], [13, 12, 13, 2, 13, 13]
    c = Case(lens, 13, H, Hkv, 128, fmt, new=new, seed=2)
    rows = []
    for b, n in enumerate(lens):
        for g in range(Hkv):
            pages = (n + new[b] + PAGE - 1) // PAGE
            keep = np.flatnonzero(rng.random(pages) < 0.4).tolist()
            if (b + g) % 3 == 0:
                keep = [j for j in keep if j < n // PAGE]
            rows.append([] if b == 1 else keep)
    o, lse = c.run(sa, rows)
    assert int(c.st.item()) == 0
    c.check(o, lse, rows)


@pytest.mark.parametrize("H", [4, 48])
def test_bad_routes_are_reported_and_left_out(sa, H):
    c = Case([640, 640, 640], 4, H, 1, 64, "bf16", seed=8)
    for rows, kept in (([[0, 3, 3, 5], [1], [2]], [[0, 3, 5], [1], [2]]),
                       ([[0, 900, 2], [1], [-5, 4]], [[0], [1], [4]]),
                       ([[5, 3, 9], [], [0, 1]], [[5, 9], [], [0, 1]])):
        o, lse = c.run(sa, rows)
        assert int(c.st.item()) == sa.SA_DEV_BAD_ROUTE
        c.check(o, lse, kept)
    # spans outside the list: nothing but the pages with new tokens
    rp = dev([0, 5, 2, 4])
    o, lse = c.run(sa, row_ptr=rp, col_idx=dev([0, 1, 2, 3]))
    assert int(c.st.item()) == sa.SA_DEV_BAD_ROUTE
    c.check(o, lse, [[], [], [2, 3]])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("base", [100, 600, 1400])
def test_runs_of_many_steps_that_end_in_new_tokens(sa, base, fmt, D):
    """Runs that hold the ends of units behind other steps, what lies behind the last tokens
    being no number, with the cache in L2 and not; every time the same."""
    c = Case([base, base + 60, base + 1, base, base - 37], 64, 48, 2, D, fmt, seed=base)
    o, lse = c.run(sa)
    c.check(o, lse)
    o, lse = o.clone(), lse.clone()
    large = torch.zeros(1 << 26, device="cuda")
    for i in range(12):
        if i % 2:
            large.add_(1)
        o2, lse2 = c.run(sa)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("H", [4, 48])
def test_bad_lengths_pages_and_parents(sa, H):
    c = Case([100, 200, 70, 300], 6, H, 2, 64, "bf16", seed=4, max_pages=5, garbage=False)
    c.table[1, 1] = c.n_pages + 7
    c.table[2, 1] = -3                        # every new token of the sequence lies there
    o, lse = c.run(sa)
    assert int(c.st.item()) == sa.SA_DEV_BAD_CACHE
    c.check(o, lse)
    c = Case([100, 200, 0], 6, H, 2, 64, "bf16", seed=4, max_pages=4, garbage=False)
    c.lens = [-4, 200, 0]
    o, lse = c.run(sa)
    assert int(c.st.item()) == sa.SA_DEV_BAD_CACHE
    c.check(o, lse)
    # no place for some, or all, new tokens
    c = Case([253, 256, 250], 6, H, 2, 64, "bf16", seed=4, max_pages=4, garbage=False)
    o, lse = c.run(sa)
    assert int(c.st.item()) == sa.SA_DEV_CAPACITY
    c.check(o, lse)
    # parents that do not come before: -1; those of tokens that do not count are not looked at
    c = Case([100, 30], 6, H, 2, 64, "bf16", new=[6, 3], seed=4)
    c.parents = np.array([[-1, 1, 0, 9, -7, 3], [-1, 0, 0, 99, 99, 99]], dtype=np.int32)
    o, lse = c.run(sa)
    assert int(c.st.item()) == sa.SA_DEV_BAD_TREE
    c.check(o, lse)
    c.parents[0] = [-1, 0, 0, 2, -1, 3]
    o, lse = c.run(sa)
    assert int(c.st.item()) == 0
    c.check(o, lse)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("H", [2, 6, 40, 60])
def test_what_a_token_does_not_see_has_no_effect(sa, H, fmt, D):
    """NaN and infinities in the keys and values of other branches."""
    S = 20
    up = np.array([[-1] + [0 if s < 4 else s - 3 for s in range(1, S)]] * 2, dtype=np.int32)
    for base in (130, 60):
        for caches in (("vc",), ("kc",), ("kc", "vc")):
            c = Case([base, base + 5], S, H, 2, D, fmt, parents=up, seed=6)
            for b in range(2):
                c.put(b, base + 5 * b + 2, base + 5 * b + 3, float("nan"), caches)
                c.put(b, base + 5 * b + 9, base + 5 * b + 10, float("inf"), caches)
            o, lse = c.run(sa)
            assert int(c.st.item()) == 0
            got = torch.isfinite(o).all(-1).all(-1).cpu().numpy()        # [B, S]
            sees = ancestors_ref(up[0], S)
            clean = ~(sees[:, 2] | sees[:, 9])
            assert got[:, clean].all()
            if "kc" not in caches:
                c.check(o, lse)
            else:                                  # the tokens that see neither, as without them
                before = o.clone()
                for b in range(2):
                    for at in (base + 5 * b + 2, base + 5 * b + 9):
                        page = int(c.table[b, at // PAGE])
                        for t in (c.kc, c.vc):
                            (t if fmt == "bf16" else t.view(torch.uint8))[page, :, at % PAGE] = 0
                after, _ = c.run(sa)
                ok = torch.from_numpy(clean).cuda()
                assert torch.equal(before[:, ok], after[:, ok])


def test_infinite_values_that_are_seen(sa):
    c = Case([70], 3, 40, 1, 64, "bf16", parents=np.array([[-1, 0, 0]], dtype=np.int32), seed=6)
    c.put(0, 71, 72, float("inf"), ("vc",))
    o, lse = c.run(sa)
    assert torch.isinf(o[0, 1]).all() and torch.isfinite(o[0, [0, 2]].float()).all()
    c.check(o, lse)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("H", [4, 40])
def test_pages_beyond_32_bit_offsets(sa, fmt, H):
    """A pool of more than 2^31 elements, its used pages at both ends."""
    D, Hkv, S = 128, 2, 5
    n_pages = (1 << 31) // (Hkv * PAGE * D) + 300
    dt = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
    c = Case([400, 64], S, H, Hkv, D, fmt, seed=13, garbage=False)
    small = [c.kc, c.vc]
    big = [torch.zeros((n_pages, Hkv, PAGE, D), dtype=dt, device="cuda") for _ in range(2)]
    where = np.array([n_pages - 1 - i if i % 2 else i for i in range(c.n_pages)])
    raw = (lambda t: t) if fmt == "bf16" else (lambda t: t.view(torch.uint8))
    for s_, b_ in zip(small, big):
        raw(b_)[dev(where, torch.int64)] = raw(s_)
    o, lse = c.run(sa)
    o, lse = o.clone(), lse.clone()
    c.table = np.where(c.table >= 0, where[np.maximum(c.table, 0)], -1)
    c.kc, c.vc = big
    o2, lse2 = c.run(sa)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("H", [4, 40])
def test_strided_queries_outputs_and_table(sa, H):
    c = Case([300, 64], 5, H, 2, 64, "bf16", seed=10)
    o, lse = c.run(sa)
    wide = torch.zeros((2, 7, H + 3, 96), dtype=torch.bfloat16, device="cuda")
    q = wide[:, 1:6, 2:H + 2, 16:80]
    q.copy_(c.q)
    buf = torch.full((5, 2, H + 1, 80), 3.0, dtype=torch.bfloat16, device="cuda")
    out = buf.permute(1, 0, 2, 3)[:, :, :H, 8:72]
    table = torch.full((2, c.max_pages + 9), -1, dtype=torch.int32, device="cuda")
    table[:, :c.max_pages] = dev(c.table)
    sa.sa_attn_tree(q, c.kc, c.vc, table[:, :c.max_pages], dev(c.lens), parents=dev(c.parents), o=out)
    torch.cuda.synchronize()
    assert torch.equal(out, o)
    assert bool((buf[:, :, H] == 3.0).all()) and bool((buf[..., :8] == 3.0).all())


@pytest.mark.parametrize("H,fmt", [(4, "bf16"), (40, "bf16"), (40, "fp8")])
def test_repeats_captured_and_on_other_streams(sa, H, fmt):
    c = Case([3000, 64, 777], 6, H, 2, 128, fmt, seed=11)
    o, lse = c.run(sa)
    o, lse = o.clone(), lse.clone()
    p = sa.make_cache_params(dev(c.table), q=c.q.cuda(), k_cache=c.kc, v_cache=c.vc)
    n = sa.sa_attn_tree_workspace_bytes(p)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")          # no care what it held
    for _ in range(3):
        o2, lse2 = c.run(sa, workspace=ws)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert c.run(sa, lse=None, want_lse=False)[1] is None
    # captured, replayed after the lengths and the tree have changed
    args = dict(q=c.q.cuda(), table=dev(c.table), lens=dev(c.lens), up=dev(c.parents))
    scale = {} if fmt == "bf16" else dict(k_scale=c.ks.cuda(), v_scale=c.vs.cuda())
    out, l2 = torch.zeros_like(o), torch.zeros_like(lse)
    call = lambda: sa.sa_attn_tree(args["q"], c.kc, c.vc, args["table"], args["lens"],
                                   parents=args["up"], o=out, lse=l2, workspace=ws, **scale)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    torch.cuda.synchronize()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, o) and torch.equal(l2, lse)
    c.lens = [2000, 10, 0]
    c.parents = random_parents(3, 6, np.random.default_rng(5))
    args["lens"].copy_(dev(c.lens))
    args["up"].copy_(dev(c.parents))
    graph.replay()
    torch.cuda.synchronize()
    fresh, flse = c.run(sa)
    assert torch.equal(out, fresh) and torch.equal(l2, flse)
    # a stream given by hand
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    o3, _ = sa.sa_attn_tree(args["q"], c.kc, c.vc, args["table"], args["lens"], parents=args["up"],
                            stream=other, **scale)
    other.synchronize()
    assert torch.equal(o3, fresh)


@pytest.mark.parametrize("H,fmt", [(4, "bf16"), (4, "fp8"), (40, "bf16"), (40, "fp8")])
def test_queries_that_are_no_numbers_stay_in_their_rows(sa, H, fmt):
    """NaN and infinities in one token's queries are its own affair, and so is their size."""
    c = Case([500, 70], 9, H, 2, 128, fmt, seed=21)
    o, lse = c.run(sa)
    o, lse = o.clone(), lse.clone()
    c.q[0, 3, 0, 5] = float("nan")
    c.q[0, 5, H - 1] = float("inf")
    c.q[1, 8, H // 2, ::2] = 3e38
    c.q[1, 0, 1] = 0.0
    c.q[1, 1, 1] = 1e-38
    o2, lse2 = c.run(sa)
    same = torch.ones((2, 9, H), dtype=torch.bool, device="cuda")
    for b, s, h in ((0, 3, 0), (0, 5, H - 1), (1, 8, H // 2), (1, 0, 1), (1, 1, 1)):
        same[b, s, h] = False
    assert torch.equal(o[same], o2[same])
    assert torch.equal(lse.transpose(1, 2)[same], lse2.transpose(1, 2)[same])
    assert bool(o2[0, 3, 0].isnan().all())
    # queries of 0: the mean of the values that are seen, lse = log of their number
    seen = [70 + 1, 70 + 1 + (1 if c.parents[1, 1] == 0 else 0)]
    for s in (0, 1):
        n = seen[s]
        off = n * 2.0 ** -24 + 2.0 ** -22 * (math.log(n) + 2)
        assert abs(float(lse2[1, 1, s]) - math.log(n)) <= off


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("H", [4, 40])
def test_the_smallest_scales(sa, H, fmt):
    """A subnormal scale makes every weight one, of what a token sees."""
    c = Case([500, 70], 9, H, 2, 128, fmt, seed=22, scale=1e-40)
    o, lse = c.run(sa)
    c.check(o, lse)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("lens,H,Hkv,S", [([2617] * 8, 56, 1, 64), ([4164, 23, 1, 361, 1803, 1019, 4693], 40, 1, 48),
                                          ([1782, 2178, 323, 39, 69, 37], 56, 8, 64)])
def test_the_same_every_time(sa, lens, H, Hkv, S, fmt, D):
    """Some hundred calls with the cache in L2 and not: loads that come early or late."""
    c = Case(lens, S, H, Hkv, D, fmt, seed=7)
    args = [c.q.cuda(), c.kc, c.vc, dev(c.table), dev(c.lens)]
    kw = {} if c.ks is None else dict(k_scale=c.ks.cuda(), v_scale=c.vs.cuda())
    p = sa.make_cache_params(args[3], q=args[0], k_cache=c.kc, v_cache=c.vc)
    kw.update(parents=dev(c.parents),
              workspace=torch.empty(sa.sa_attn_tree_workspace_bytes(p), dtype=torch.uint8, device="cuda"))
    large = torch.zeros(1 << 26, device="cuda")
    o, lse = sa.sa_attn_tree(*args, **kw)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(300):
        if i % 2:
            large.add_(1)
        o2, lse2 = sa.sa_attn_tree(*args, **kw)
        differ += (o2 != o).any().long() + (lse2 != lse).any().long()
    assert int(differ.item()) == 0
    if fmt == "bf16" and D == 64 and Hkv == 8:
        c.check(o, lse)


def test_calls_side_by_side(sa):
    """Calls on two streams at once, each with its own workspace, as one by one."""
    cases = [Case([4000, 900], 6, H, 2, 128, fmt, seed=30 + i)
             for i, (H, fmt) in enumerate([(4, "bf16"), (40, "fp8"), (40, "bf16"), (12, "fp8")])]
    alone = [tuple(x.clone() for x in c.run(sa)) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    args = [dict(q=c.q.cuda(), table=dev(c.table), lens=dev(c.lens), up=dev(c.parents),
                 kw={} if c.ks is None else dict(k_scale=c.ks.cuda(), v_scale=c.vs.cuda()))
            for c in cases]
    torch.cuda.synchronize()
    outs = [[] for _ in cases]
    for _ in range(5):
        for i, (c, a, st) in enumerate(zip(cases, args, streams)):
            with torch.cuda.stream(st):
                outs[i].append(sa.sa_attn_tree(a["q"], c.kc, c.vc, a["table"], a["lens"],
                                               parents=a["up"], **a["kw"]))
    torch.cuda.synchronize()
    for (o, lse), got in zip(alone, outs):
        for o2, l2 in got:
            assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_one_token_is_a_decoding_step(sa):
    """With one new token the tree is sa_attn_decode over the length with it."""
    c = Case([300, 0, 64, 1000], 1, 8, 2, 128, "bf16", seed=3)
    o, lse = c.run(sa)
    d, dl = sa.sa_attn_decode(c.q.cuda(), c.kc, c.vc, dev(c.table), dev([n + 1 for n in c.lens]))
    assert torch.equal(o, d) and torch.equal(lse, dl)


def test_the_binding_refuses_what_does_not_fit(sa):
    c = Case([100, 64], 5, 4, 2, 64, "bf16", seed=1)
    q, t, n = c.q.cuda(), dev(c.table), dev(c.lens)
    ok = lambda **kw: sa.sa_attn_tree(q, c.kc, c.vc, t, n, **kw)
    ok()
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    for kw in (dict(parents=i(2, 4)), dict(parents=i(4)), dict(parents=i(3, 5)),
               dict(parents=i(2, 5).long()), dict(parents=i(2, 5).cpu()), dict(parents=i(5, 2).t()),
               dict(new_lens=i(3)), dict(row_ptr=i(5)), dict(row_ptr=i(4), col_idx=i(2)),
               dict(lse=torch.zeros(2, 4, device="cuda")), dict(o=q[:, :4]),
               dict(o=torch.zeros_like(q).float()), dict(k_scale=i(2))):
        with pytest.raises((ValueError, sa.SaError)):
            ok(**kw)
    with pytest.raises(sa.SaError):
        ok(o=q)
    with pytest.raises(sa.SaError):
        ok(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(sa.SaError):
        sa.sa_attn_tree(torch.zeros((1, 65, 4, 64), dtype=torch.bfloat16, device="cuda"), c.kc, c.vc,
                        t[:1], n[:1])
    torch.cuda.synchronize()
