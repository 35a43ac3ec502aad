"""sa_route_pages: its lists equal those of scores in fp64, and sa_cache_append,
sa_route_pages and sa_attn_decode run together as a decoding loop."""

import math

import numpy as np
import pytest
import torch

import oracle
from cache_helpers import PAGE, dev, new_cache, page_table, status, values
from helpers import lib
from oracle.cache_oracle import decode_ref, route_pages_ref, turn_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return lib()


class Case:
    def __init__(self, lens, H, Hkv, D, seed=0, qmag=1.0, max_pages=None):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.Hkv, self.D = lens, H, Hkv, D
        self.max_pages = max_pages or max(1, max((n + PAGE - 1) // PAGE for n in lens))
        self.n_pages = sum((max(n, 0) + PAGE - 1) // PAGE for n in lens) + 1
        self.table = page_table(lens, self.max_pages, self.n_pages, gen)
        self.q = (qmag * torch.randn((len(lens), 1, H, D), generator=gen)).to(torch.bfloat16)
        self.ksum = 8 * torch.randn((self.n_pages, Hkv, D), generator=gen)

    def run(self, sa, prefix, budget, cap=None, **kw):
        self.st = status()
        if cap is not None:
            kw["col_idx"] = torch.full((cap + 4,), -9, dtype=torch.int32, device="cuda")[:cap]
        rp, ci = sa.sa_route_pages(self.q.cuda(), self.ksum.cuda(), dev(self.table),
                                   dev(self.lens), prefix, budget, dev_status=self.st, **kw)
        torch.cuda.synchronize()
        return rp.cpu().numpy(), ci.cpu().numpy()

    def check(self, rp, ci, prefix, budget):
        want = route_pages_ref(self.q[:, 0].double().numpy(), self.ksum.numpy(), self.table,
                               self.lens, prefix, budget)
        assert rp[0] == 0 and np.array_equal(np.diff(rp), [len(r) for r in want])
        for r, pages in enumerate(want):
            assert ci[rp[r]:rp[r + 1]].tolist() == pages, r


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (8, 8), (7, 1), (56, 8), (56, 1), (100, 1), (16, 1)])
@pytest.mark.parametrize("lens,prefix,budget", [
    ([0], 0, 4), ([1], 951, 4), ([64], 0, 0), ([65], 64, 1), ([4000, 10, 0, 2000], 100, 12),
    ([9000], 951, 8), ([9000, 4097], 0, 10000), ([3333] * 9, 65, 20)])
def test_lists_equal_the_definition(sa, lens, prefix, budget, H, Hkv, D):
    c = Case(lens, H, Hkv, D, seed=len(lens) + H + D)
    rp, ci = c.run(sa, prefix, budget)
    assert int(c.st.item()) == 0
    c.check(rp, ci, prefix, budget)


@pytest.mark.parametrize("seed", range(4))
def test_scores_that_nearly_tie(sa, seed):
    """Pages whose sums differ in the last bits only: fp32 sums cannot tell
    them apart, the list must."""
    c = Case([64 * 300, 64 * 40], 8, 2, 128, seed=seed)
    base = c.ksum[:1].clone()
    gen = torch.Generator().manual_seed(seed)
    c.ksum = base * (1 + 2.0 ** -22 * torch.randint(-4, 5, c.ksum.shape, generator=gen))
    rp, ci = c.run(sa, 64, 20)
    c.check(rp, ci, 64, 20)


@pytest.mark.parametrize("scale", [1e-30, 1e-18, 1e15, 1e30])
def test_near_ties_of_very_small_and_large_sums(sa, scale):
    """The error bound neither vanishes nor overflows with the sums' size."""
    c = Case([64 * 300, 64 * 40], 8, 2, 64, seed=7)
    gen = torch.Generator().manual_seed(7)
    c.ksum = c.ksum[:1] * (1 + 2.0 ** -22 * torch.randint(-4, 5, c.ksum.shape, generator=gen)) * scale
    rp, ci = c.run(sa, 64, 20)
    c.check(rp, ci, 64, 20)


@pytest.mark.parametrize("qmag", [1e-35, 1e-20, 1.0, 1e30])
@pytest.mark.parametrize("scale", [1e-41, 1e-36, 1e-26])
def test_near_ties_next_to_the_least_floats(sa, scale, qmag):
    """Sums, queries and products that fp32 or bf16 hold in part or not at all;
    a row of 300 pages and one of 40, which are ranked differently."""
    c = Case([64 * 300, 64 * 40], 8, 2, 64, seed=8, qmag=qmag)
    gen = torch.Generator().manual_seed(8)
    c.ksum = c.ksum[:1] * (1 + 2.0 ** -22 * torch.randint(-4, 5, c.ksum.shape, generator=gen)) * scale
    for budget in (3, 20):
        rp, ci = c.run(sa, 64, budget)
        c.check(rp, ci, 64, budget)


def test_pages_of_very_unlike_sizes(sa):
    """Sums between 1e-42 and 1e3 in one row."""
    for seed, qmag in enumerate((1.0, 1e-10, 1e20)):
        c = Case([64 * 400], 4, 2, 128, seed=seed, qmag=qmag)
        gen = torch.Generator().manual_seed(seed)
        c.ksum = c.ksum * 10.0 ** -(43 * torch.rand((c.n_pages, 1, 1), generator=gen))
        for budget in (2, 50, 200, 330):
            rp, ci = c.run(sa, 0, budget)
            c.check(rp, ci, 0, budget)


@pytest.mark.parametrize("n_pages", [40, 250, 2100])
def test_clusters_of_near_ties(sa, n_pages):
    """Scores that differ from one part in 16 to the last bits: some pages are
    decided by the error bound, some by the ranks within it, some exactly."""
    c = Case([64 * n_pages, 64 * 70], 12, 2, 128, seed=n_pages)
    gen = torch.Generator().manual_seed(n_pages)
    step = 2.0 ** -torch.randint(4, 24, (c.n_pages, 1, 1), generator=gen)
    c.ksum = c.ksum[:1] * (1 + step * torch.randint(-2, 3, (c.n_pages, 1, 1), generator=gen))
    for budget in (2, 9, 20, 33, 60, n_pages // 2, n_pages - 3):
        rp, ci = c.run(sa, 64, budget)
        c.check(rp, ci, 64, budget)


@pytest.mark.parametrize("n_pages", [30, 700, 5000])
def test_rows_of_zeros_keep_the_first_pages(sa, n_pages):
    c = Case([64 * n_pages, 64 * 90], 4, 2, 64, seed=9)
    c.q[0] = 0.0
    c.q[1, :, 2:] = -0.0
    for budget in (1, 2, 17, n_pages - 2):
        rp, ci = c.run(sa, 65, budget)
        c.check(rp, ci, 65, budget)
    c.table[0, 3] = -1                                 # one page that is not there
    rp, ci = c.run(sa, 65, 17)
    c.check(rp, ci, 65, 17)


def test_equal_scores_go_to_the_lower_page(sa):
    c = Case([64 * 500], 4, 2, 64, seed=1)
    c.ksum[:] = c.ksum[0]
    rp, ci = c.run(sa, 0, 7)
    c.check(rp, ci, 0, 7)
    assert ci[:7].tolist() == [0, 1, 2, 3, 4, 5, 499]
    c.ksum[:] = 0.0                                    # +0 and -0 are equal
    c.ksum[::2] = -0.0
    rp, ci = c.run(sa, 0, 7)
    c.check(rp, ci, 0, 7)


def test_scores_that_are_no_numbers(sa):
    c = Case([64 * 100], 4, 2, 64, seed=2)
    t = c.table[0]
    c.ksum[t[3]], c.ksum[t[4], 0, 5], c.ksum[t[9], 1, 0] = float("nan"), float("nan"), float("inf")
    c.ksum[t[20]] = 3e38                               # overflows fp32, not fp64
    c.ksum[t[21]] = 2.9e38
    for budget in (5, 98, 99, 100):
        rp, ci = c.run(sa, 0, budget)
        c.check(rp, ci, 0, budget)
    c.q[:] = float("nan")
    rp, ci = c.run(sa, 0, 5)
    c.check(rp, ci, 0, 5)


def test_bad_lengths_and_pages(sa):
    c = Case([1000, 640, 700], 4, 2, 64, seed=3)
    c.table[0, 4], c.table[1, 2] = -1, c.n_pages
    rp, ci = c.run(sa, 0, 6)
    assert int(c.st.item()) == sa.SA_DEV_BAD_CACHE
    c.check(rp, ci, 0, 6)
    c.lens = [10 ** 7, -4, 700]
    c.table[0] = np.arange(16) % c.n_pages
    rp, ci = c.run(sa, 0, 6)
    assert int(c.st.item()) == sa.SA_DEV_BAD_CACHE
    c.check(rp, ci, 0, 6)


def test_a_short_list_is_cut_and_reported(sa):
    c = Case([1000, 640], 4, 2, 64, seed=4)
    full_rp, full_ci = c.run(sa, 64, 6)
    rp, ci = c.run(sa, 64, 6, cap=15)
    assert int(c.st.item()) == sa.SA_DEV_CAPACITY
    assert np.array_equal(rp, full_rp) and np.array_equal(ci, full_ci[:15])


def test_many_rows_and_a_dirty_workspace(sa):
    lens = [(131 * i) % 2000 for i in range(300)]
    c = Case(lens, 8, 4, 64, seed=5)
    p = sa.make_cache_params(dev(c.table), q=c.q.cuda(), k_sum=c.ksum.cuda(), prefix_len=64,
                             budget=9)
    ws = torch.full((sa.sa_route_pages_workspace_bytes(p),), 0xFF, dtype=torch.uint8, device="cuda")
    rp, ci = c.run(sa, 64, 9, workspace=ws)
    c.check(rp, ci, 64, 9)


@pytest.mark.parametrize("n_pages", [3000, 9000])
def test_long_sequences(sa, n_pages):
    c = Case([64 * n_pages - 5, 64 * 1200], 4, 1, 64, seed=n_pages)
    rp, ci = c.run(sa, 951, 300)
    assert int(c.st.item()) == 0
    c.check(rp, ci, 951, 300)


def test_rows_beyond_32_bit_offsets(sa):
    """Key sums of a pool of 5 GB, the sequence's pages at its end."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    c = Case([64 * 40 - 3], 8, 8, 128, seed=23)
    n = 1_250_000
    big = torch.empty((n, 8, 128), device="cuda")
    big[n - c.n_pages:] = c.ksum.cuda()
    table = dev(c.table) + (n - c.n_pages)
    st = status()
    rp, ci = sa.sa_route_pages(c.q.cuda(), big, table, dev(c.lens), 64, 9, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    c.check(rp.cpu().numpy(), ci.cpu().numpy(), 64, 9)


def test_streams_and_refusals(sa):
    c = Case([4000, 640], 4, 2, 64, seed=24)
    q, k, t, l = c.q.cuda(), c.ksum.cuda(), dev(c.table), dev(c.lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        rp, ci = sa.sa_route_pages(q, k, t, l, 64, 9, stream=stream)
        torch.cuda.synchronize()
        c.check(rp.cpu().numpy(), ci.cpu().numpy(), 64, 9)
    ok = dict(q=q, k_sum=k, page_table=t, seq_lens=l, prefix_len=64, budget=9)
    for bad in (dict(q=q.float()), dict(k_sum=k.half()), dict(k_sum=k[:, :, :32]), dict(k_sum=k[0]),
                dict(q=q[:, 0]), dict(seq_lens=l[:1]), dict(budget=1 << 40), dict(budget="x"),
                dict(row_ptr=dev([0] * 4)), dict(col_idx=torch.zeros(99, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            sa.sa_route_pages(**{**ok, **bad})
    for bad, code in ((dict(budget=-1), 1), (dict(prefix_len=-1), 1), (dict(q=q.expand(2, 1, 4, 64)[:, :, :3]), 1)):
        with pytest.raises(sa.SaError) as e:
            sa.sa_route_pages(**{**ok, **bad, "row_ptr": dev([0] * 5), "col_idx": dev([0] * 99),
                                 "workspace": torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")})
        assert e.value.code == code
    torch.cuda.synchronize()


# ------------------------------------------------------------- run together --

@pytest.mark.parametrize("fmt,rope,D", [("bf16", "interleaved", 128), ("fp8", "half", 64)])
def test_a_decoding_loop(sa, fmt, rope, D):
    """A prompt, then token after token: append, route, attend, as one captured
    step that reads and writes the lengths on the device."""
    B, H, Hkv, prompt, steps, budget, prefix = 3, 6, 2, 200, 5, 3, 64
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16).cuda()
    max_pages, n_pages = 5, 17
    table = page_table([64 * max_pages] * B, max_pages, n_pages, gen)
    kc, _ = new_cache(n_pages, Hkv, D, fmt)
    vc, _ = new_cache(n_pages, Hkv, D, fmt)
    ksum = torch.full((n_pages, Hkv, D), float("nan"), device="cuda")
    sc = torch.full((Hkv,), 0.02, device="cuda") if fmt == "fp8" else None
    ang = torch.arange(64 * max_pages)[:, None] * 10000.0 ** (-torch.arange(D // 2) / (D // 2))
    cos, sin = ang.cos().cuda(), ang.sin().cuda()
    gq, gk = (1 + 0.1 * torch.randn(D, generator=gen)).cuda(), (1 + 0.1 * torch.randn(D, generator=gen)).cuda()
    turn = dict(qk_norm=True, gamma_q=gq, gamma_k=gk, cos=cos, sin=sin, rope=rope, k_scale=sc,
                v_scale=sc, k_sum=ksum)
    st, lens = status(), torch.zeros(B, dtype=torch.int32, device="cuda")
    lens2 = torch.zeros_like(lens)
    new = torch.tensor([prompt, 64, 1], dtype=torch.int32, device="cuda")
    tbl = dev(table)
    ks, vs = [r(B, prompt, Hkv, D)], [r(B, prompt, Hkv, D)]
    sa.sa_cache_append(ks[0], vs[0], kc, vc, tbl, lens, new_lens=new, lens_out=lens2,
                       dev_status=st, **turn)
    lens.copy_(lens2)
    k1, v1, q1 = (torch.empty((B, 1, h, D), dtype=torch.bfloat16, device="cuda") for h in (Hkv, Hkv, H))

    def step():
        q = sa.sa_cache_append(k1, v1, kc, vc, tbl, lens, q=q1, lens_out=lens2, dev_status=st, **turn)
        rp, ci = sa.sa_route_pages(q, ksum, tbl, lens2, prefix, budget, dev_status=st)
        o, lse = sa.sa_attn_decode(q, kc, vc, tbl, lens2, row_ptr=rp, col_idx=ci, k_scale=sc,
                                   v_scale=sc, dev_status=st)
        lens.copy_(lens2)
        return q, rp, ci, o, lse

    graph = None
    for i in range(steps):
        for t, h in ((k1, Hkv), (v1, Hkv), (q1, H)):
            t.copy_(r(B, 1, h, D))
        if i == 0:
            out = step()
        else:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    out = step()
            graph.replay()
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        q, rp, ci, o, lse = (t.cpu() for t in out)
        n = [prompt + i + 1, 64 + i + 1, 1 + i + 1]
        assert lens.tolist() == n
        # the appended query and the newest key, from their definitions
        for b in range(B):
            c, s = cos[n[b] - 1].cpu().double().numpy(), sin[n[b] - 1].cpu().double().numpy()
            y, mag = turn_ref(q1[b, 0].cpu().double().numpy(), gq.cpu().double().numpy(), 1e-6, c, s, rope)
            assert np.all(np.abs(q[b, 0].double().numpy() - y) <= 2.0 ** -8 * np.abs(y) + 2e-6 * mag)
        qn = q[:, 0].double().numpy()
        rows = route_pages_ref(qn, ksum.cpu().numpy(), table, n, prefix, budget)
        for k, pages in enumerate(rows):
            assert ci[int(rp[k]):int(rp[k + 1])].tolist() == pages
        eo, el, mag = decode_ref(qn, values(kc, sc), values(vc, sc), table, n, 1 / math.sqrt(D), rows)
        got = o[:, 0].double().numpy()
        # logits of at most |q||k| / sqrt(D) < 20: dl < 1e-4
        assert np.all(np.abs(got - eo) <= 2.0 ** -8 * np.abs(eo) + (2e-4 + 2.0 ** -11) * mag)
        assert np.all(np.abs(lse[..., 0].double().numpy() - el) <= 2e-4)


def test_every_page_gives_the_dense_layer(sa):
    """One bidirectional prefix through sa_qk_prologue and sa_attn_dense, the
    same tokens cached: the newest token's row agrees with the cache's."""
    S, H, D = 500, 3, 128
    gen = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn((1, S, H, D), generator=gen).to(torch.bfloat16).cuda() for _ in range(3))
    ang = torch.arange(S)[:, None] * 10000.0 ** (-torch.arange(D // 2) / (D // 2))
    cos, sin = ang.cos().cuda(), ang.sin().cuda()
    qo, ko, _ = sa.sa_qk_prologue(q, k, eps=1e-6, cos=cos, sin=sin)
    dense, dl = sa.sa_attn_dense(qo, ko, v)
    table = dev(page_table([S], 8, 9, gen))
    kc, _ = new_cache(9, H, D, "bf16")
    vc, _ = new_cache(9, H, D, "bf16")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    q2 = sa.sa_cache_append(k, v, kc, vc, table, lens, q=q, qk_norm=True, cos=cos, sin=sin)
    o, lse = sa.sa_attn_decode(q2[:, -1:], kc, vc, table, lens + S)
    torch.cuda.synchronize()
    # one rotation, one norm, one rounding each: at most an element in a thousand differs
    assert float((q2 != qo).float().mean()) < 1e-3
    assert float((values(kc)[table[0, :8].cpu().numpy()].transpose(0, 2, 1, 3).reshape(-1, H, D)[:S]
                  != ko[0].float().cpu().numpy()).mean()) < 1e-3
    ref = dense[:, -1:].float()
    # both are within half a bf16 step of nearly the same value; sa_attn_dense rounds P and V to fp16
    assert float((o.float() - ref).abs().max()) <= 2.0 ** -7 * float(ref.abs().max()) + 1e-3
    assert float((lse[0, :, 0] - dl[0, :, -1]).abs().max()) <= 2e-3


def test_the_oracle_of_routes_ranks_like_the_layers_router(sa):
    """For full pages the sums rank as the block means of the layer's router do."""
    S, D = 640, 64
    gen = torch.Generator().manual_seed(5)
    q, k = (torch.randn((1, S, 1, D), generator=gen).to(torch.bfloat16) for _ in range(2))
    sums = k.double().reshape(10, 64, 1, D).sum(1)
    rows = route_pages_ref(q[:, -1].double().numpy(), sums.numpy(), np.arange(10)[None], [S], 0, 4)
    means = (k.double().reshape(10, 64, D).mean(1) @ q[0, -1, 0].double()).numpy()
    best = sorted(np.argsort(-means[:9])[:3].tolist() + [9])
    assert rows[0] == best and oracle.BLOCK == PAGE
