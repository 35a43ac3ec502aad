"""sa_attn_decode against the fp64 definition.

Bounds, from the arithmetic. A logit's products are exact in fp32 and summed
with an error of at most (D + 4) 2^-24 of scale sum |q k|; its scaling, the
subtraction of the maximum and the exponential add 2^-22 of the logit's and of
one part: dl. A weight is rounded to 2^-16 of itself (2^-11 in fp16), the sums
of n weights in fp32 are off by at most n 2^-24. So
  |o - exact| <= 2^-8 |exact| + (2 dl + 2^-11 or 2^-16 + 2 n 2^-24) sum a |v|,
  |lse - exact| <= dl + n 2^-24 + 2^-22 (|lse| + 1)."""

import math

import numpy as np
import pytest
import torch

from cache_helpers import PAGE, dev, new_cache, page_table, status, values
from helpers import lib
from oracle.cache_oracle import decode_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return lib()


class Case:
    def __init__(self, lens, H, Hkv, D, fmt, layout="page_head", scale=0.0, qmag=2.0, seed=0,
                 max_pages=None, garbage=True):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.Hkv, self.D, self.fmt, self.scale = lens, H, Hkv, D, fmt, scale
        B = len(lens)
        need = [(max(n, 0) + PAGE - 1) // PAGE for n in lens]
        self.max_pages = max_pages or max(1, max(need))
        self.n_pages = sum(min(x, self.max_pages) for x in need) + 2
        self.table = page_table(lens, self.max_pages, self.n_pages, gen)
        self.q = (qmag * torch.randn((B, 1, H, D), generator=gen)).to(torch.bfloat16)
        fill = 1.0 if fmt == "bf16" else 40.0
        self.kc, _ = new_cache(self.n_pages, Hkv, D, fmt, layout, fill, gen)
        self.vc, _ = new_cache(self.n_pages, Hkv, D, fmt, layout, fill, gen)
        self.ks = self.vs = None
        if fmt == "fp8":
            self.ks = 0.01 + 0.03 * torch.rand(Hkv, generator=gen)
            self.vs = 0.01 + 0.03 * torch.rand(Hkv, generator=gen)
        if garbage:                    # what lies behind a sequence's last token has no effect
            for b, n in enumerate(lens):
                if n % PAGE and 0 < n <= PAGE * self.max_pages:
                    page = int(self.table[b, n // PAGE])
                    for t in (self.kc, self.vc):
                        u = t if fmt == "bf16" else t.view(torch.uint8)
                        bad = float("nan") if fmt == "bf16" else 0x7F
                        u[page, :, n % PAGE:] = bad
                        if fmt == "bf16" and n % PAGE < 62:
                            u[page, :, n % PAGE + 1] = float("inf")

    def run(self, sa, rows=None, **kw):
        c = lambda t: None if t is None else t.cuda()
        self.st = status()
        args = dict(scale=self.scale, k_scale=c(self.ks), v_scale=c(self.vs), dev_status=self.st)
        if rows is not None:
            rp = np.concatenate([[0], np.cumsum([len(r) for r in rows])])
            ci = np.concatenate([np.asarray(r, dtype=np.int64) for r in rows] + [[0]])
            args.update(row_ptr=dev(rp), col_idx=dev(ci))
        args.update(kw)
        o, lse = sa.sa_attn_decode(c(self.q), self.kc, self.vc, dev(self.table), dev(self.lens),
                                   **args)
        torch.cuda.synchronize()
        return o, lse

    def check(self, o, lse, rows=None):
        """`rows`: the pages that count."""
        scale = self.scale or 1 / math.sqrt(self.D)
        k, v = values(self.kc, self.ks), values(self.vc, self.vs)
        q = self.q[:, 0].double().numpy()
        eo, el, mag = decode_ref(q, k, v, self.table, self.lens, scale, rows)
        knorm = np.linalg.norm(np.nan_to_num(k, posinf=0, neginf=0), axis=-1).max()
        top = scale * np.linalg.norm(q, axis=-1) * knorm                    # [B, H]
        n = np.clip(np.asarray(self.lens), 0, None)[:, None]
        dl = top * ((self.D + 4) * 2.0 ** -24 + 2.0 ** -22) + 2.0 ** -22
        w = 2 * dl + (2.0 ** -16 if self.fmt == "bf16" else 2.0 ** -11) + 2 * n * 2.0 ** -24
        got = o[:, 0].cpu().double().numpy()
        tol = 2.0 ** -8 * np.abs(eo) + w[..., None] * mag
        assert np.all(np.abs(got - eo) <= tol), float(np.max(np.abs(got - eo) / np.maximum(tol, 1e-30)))
        if lse is not None:
            gl = lse[..., 0].cpu().double().numpy()
            empty = np.isneginf(el)
            assert np.array_equal(np.isneginf(gl), empty)
            tl = dl + n * 2.0 ** -24 + 2.0 ** -22 * (np.abs(np.where(empty, 0, el)) + 1)
            assert np.all(np.abs(gl[~empty] - el[~empty]) <= np.broadcast_to(tl, el.shape)[~empty])


LENS = [[0], [1], [2], [63], [64], [65], [129, 0, 1, 64], [777], [2048, 5, 700],
        [(97 * i) % 330 for i in range(40)]]
HEADS = [(1, 1), (4, 4), (5, 1), (7, 1), (16, 2), (17, 1), (32, 1), (33, 1), (56, 8), (56, 1)]


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", LENS, ids=lambda l: f"{len(l)}x{max(l)}")
def test_lengths(sa, lens, D, fmt):
    c = Case(lens, 8, 2, D, fmt, seed=len(lens) + D)
    o, lse = c.run(sa)
    assert int(c.st.item()) == 0
    c.check(o, lse)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv", HEADS)
def test_head_layouts(sa, H, Hkv, D, fmt):
    c = Case([300, 64, 17], H, Hkv, D, fmt, seed=H)
    o, lse = c.run(sa)
    assert int(c.st.item()) == 0
    c.check(o, lse)


@pytest.mark.parametrize("H,Hkv", [(65, 1), (100, 1), (130, 2), (128, 1)])
def test_many_query_heads_on_one_kv_head(sa, H, Hkv):
    c = Case([200, 64, 131], H, Hkv, 128, "bf16", seed=H)
    o, lse = c.run(sa)
    assert int(c.st.item()) == 0
    c.check(o, lse)


@pytest.mark.parametrize("layout", ["page_token", "gapped"])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
def test_cache_layouts(sa, layout, fmt, D):
    c = Case([500, 70, 64], 6, 3, D, fmt, layout=layout, seed=9)
    o, lse = c.run(sa)
    c.check(o, lse)


def test_many_rows(sa):
    """More rows than a grid of resident blocks, most of them short."""
    lens = [(53 * i) % 190 for i in range(500)]
    c = Case(lens, 4, 2, 64, "bf16", seed=5)
    c.check(*c.run(sa))


def test_long_sequence_in_a_batch_of_short_ones(sa):
    c = Case([20000] + [3] * 6 + [0, 9000], 8, 1, 128, "fp8", seed=6)
    c.check(*c.run(sa))


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_peaked_and_flat_softmax(sa, fmt):
    for qmag, scale in ((0.0, 0.0), (30.0, 0.0), (1.0, 3.0), (1.0, 1e-4)):
        c = Case([1000, 130], 8, 2, 128, fmt, qmag=qmag, scale=scale, seed=7)
        c.check(*c.run(sa))


@pytest.mark.parametrize("D", [64, 128])
def test_queries_next_to_zero(sa, D):
    """Logits that underflow are zero, in a page with masked keys too."""
    for q, ks in ((2.0 ** -133, 1e-3), (2.0 ** -126, 1e-20), (-2.0 ** -130, 0.02)):
        c = Case([65, 1000, 3], 4, 2, D, "fp8", seed=21)
        c.q.fill_(q)
        assert float(c.q.float().abs().max()) == abs(q)
        c.ks.fill_(ks)
        c.check(*c.run(sa))


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_very_large_logits_stay_finite(sa, fmt):
    """Logits whose spacing in fp32 is above one: the weights are no better
    than the logits, but none overflows."""
    for seed in range(4):
        for qmag in (1e6, 1e8, 1e12):
            c = Case([700, 64, 1], 4, 2, 64, fmt, qmag=qmag, seed=seed)
            o, lse = c.run(sa)
            assert torch.isfinite(o).all() and torch.isfinite(lse).all()
            c.check(o, lse)


def test_one_far_key_among_many_small_weights(sa):
    """A key far above the others in one page, the mass spread over the rest."""
    c = Case([6000], 4, 1, 128, "fp8", qmag=0.5, seed=8)
    q = c.q[0, 0].float().mean(0)
    code = (q / q.norm() * 300).to(torch.float8_e4m3fn).view(torch.uint8)
    c.kc.view(torch.uint8)[int(c.table[0, 40]), 0, 13] = code.cuda()
    c.check(*c.run(sa))


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_routed_pages(sa, fmt):
    lens = [700, 0, 64, 1500]
    c = Case(lens, 6, 2, 128, fmt, seed=11)
    rng = np.random.default_rng(0)
    rows = []
    for n in lens:
        nb = (n + PAGE - 1) // PAGE
        rows += [sorted(rng.choice(nb, size=min(nb, 5), replace=False).tolist()), list(range(nb))]
    rows[0] = []                       # nothing to attend for one head group
    o, lse = c.run(sa, rows)
    assert int(c.st.item()) == 0
    c.check(o, lse, rows)
    assert torch.all(o[0, 0, :3] == 0) and torch.all(torch.isneginf(lse[0, :3]))
    # every page listed: the unrouted result
    full = [list(range((n + PAGE - 1) // PAGE)) for n in lens for _ in range(2)]
    a, b = c.run(sa, full)
    x, y = c.run(sa)
    assert torch.equal(a, x) and torch.equal(b, y)


def test_bad_routes_are_reported_and_left_out(sa):
    lens = [700, 700, 700]
    c = Case(lens, 4, 2, 64, "bf16", seed=12)
    good = [[0, 3, 10], [1, 2], [4, 5], [0, 9], [7], [8, 10]]
    bad = [list(r) for r in good]
    bad[0], good[0] = [0, 3, 3, 2, 10], [0, 3, 10]       # repeated, descending
    bad[2], good[2] = [-1, 4, 5, 11, 99], [4, 5]         # outside the sequence
    o, lse = c.run(sa, bad)
    assert int(c.st.item()) == sa.SA_DEV_BAD_ROUTE
    c.check(o, lse, good)
    # row_ptr that steps back, leaves col_idx, or spans too much: those rows whole
    rp = [0, 3, 2, 4, 4, 6, 5000]
    ci = [0, 3, 10, 4, 7, 9]
    o, lse = c.run(sa, row_ptr=dev(rp), col_idx=dev(ci))
    assert int(c.st.item()) == sa.SA_DEV_BAD_ROUTE
    c.check(o, lse, [[0, 3, 10], [], [10], [], [7, 9], []])  # row 2: col_idx[2:4] = 10, 4
    rp = [-7, 2, 3, 3, 3, 3, 3]
    o, lse = c.run(sa, row_ptr=dev(rp), col_idx=dev([1, 2, 3]))
    assert int(c.st.item()) == sa.SA_DEV_BAD_ROUTE
    c.check(o, lse, [[], [3], [], [], [], []])


def test_bad_lengths_and_pages(sa):
    c = Case([300, 200, 128], 4, 2, 64, "bf16", seed=13, garbage=False)
    c.table[0, 2], c.table[1, 0] = c.n_pages, -1
    o, lse = c.run(sa)
    assert int(c.st.item()) == sa.SA_DEV_BAD_CACHE
    c.check(o, lse)                    # the oracle leaves those pages out
    c = Case([300, 200, 128], 4, 2, 64, "bf16", seed=13, garbage=False)
    c.lens = [10 ** 6, -1, 128]        # beyond the table: all it holds
    o, lse = c.run(sa)
    assert int(c.st.item()) == sa.SA_DEV_BAD_CACHE
    c.lens = [64 * c.max_pages, 0, 128]
    c.check(o, lse)


def test_not_a_number_among_valid_keys_stays_in_its_rows(sa):
    c = Case([300, 200], 4, 2, 64, "bf16", seed=14)
    c.kc[int(c.table[0, 1]), 0, 5, 3] = float("nan")
    o, lse = c.run(sa)
    assert torch.isnan(o[0, 0, :2]).all() and torch.isnan(lse[0, :2]).all()
    assert not torch.isnan(o[0, 0, 2:]).any() and not torch.isnan(o[1]).any()


def test_infinite_values_stay_infinite(sa):
    c = Case([300, 200], 4, 2, 64, "bf16", seed=19)
    c.vc[int(c.table[0, 1]), 0, 5, 3] = float("inf")
    c.vc[int(c.table[0, 2]), 0, 9, 40] = float("-inf")
    o, lse = c.run(sa)
    for h in (0, 1):
        assert o[0, 0, h, 3] == float("inf") and o[0, 0, h, 40] == float("-inf")
        assert torch.isfinite(o[0, 0, h]).sum() == 62
    assert torch.isfinite(o[0, 0, 2:]).all() and torch.isfinite(o[1]).all()
    assert torch.isfinite(lse).all()


def test_many_routed_rows(sa):
    """More rows than one warp scans, and than the grid has blocks."""
    for B, H, Hkv in ((60, 4, 2), (300, 4, 4)):
        lens = [(71 * i) % 700 for i in range(B)]
        c = Case(lens, H, Hkv, 64, "bf16", seed=20)
        rng = np.random.default_rng(B)
        rows = []
        for n in lens:
            nb = (n + PAGE - 1) // PAGE
            rows += [sorted(rng.choice(nb, size=rng.integers(0, nb + 1), replace=False).tolist())
                     for _ in range(Hkv)]
        o, lse = c.run(sa, rows)
        assert int(c.st.item()) == 0
        c.check(o, lse, rows)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_pages_beyond_32_bit_offsets(sa, fmt):
    """A pool of 5 GB whose last pages hold the sequence: bytes and elements
    past 2^32."""
    n_pages, D = (320_000, 128) if fmt == "bf16" else (640_000, 128)
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    c = Case([200, 64], 4, 1, D, fmt, seed=21)
    dt = c.kc.dtype
    big = [torch.empty((n_pages, 1, PAGE, D), dtype=dt, device="cuda") for _ in range(2)]
    far = np.array([n_pages - 1 - i for i in range(c.n_pages)])
    for t, old in zip(big, (c.kc, c.vc)):
        for i, p in enumerate(far):
            t.view(torch.uint8)[p] = old.view(torch.uint8)[i]
    small = (c.kc, c.vc, c.table)
    c.kc, c.vc = big
    c.table = np.where(c.table >= 0, far[np.maximum(c.table, 0)], -1).astype(np.int32)
    o, lse = c.run(sa)
    c.kc, c.vc, c.table = small
    c.check(o, lse)


def test_shared_pages_and_shared_table_rows(sa):
    """One prefix page in two sequences, and twice in one."""
    c = Case([128, 192], 2, 1, 64, "bf16", seed=15)
    c.table[1, 0] = c.table[0, 0]
    c.table[1, 1] = c.table[0, 0]
    c.check(*c.run(sa))


def test_strided_queries_outputs_and_table(sa):
    c = Case([300, 65], 4, 2, 128, "bf16", seed=16)
    want, lw = c.run(sa)
    wide = torch.zeros((2, 3, 9, 128), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:2, 2:6] = c.q.cuda()
    out = torch.full((2, 2, 7, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    table = torch.full((2, 9), -1, dtype=torch.int32, device="cuda")
    table[:, :c.max_pages] = dev(c.table)
    o, lse = sa.sa_attn_decode(wide[:, 1:2, 2:6], c.kc, c.vc, table[:, :c.max_pages], dev(c.lens),
                               o=out[:, 1:2, 1:5])
    torch.cuda.synchronize()
    assert torch.equal(out[:, 1:2, 1:5], want) and torch.equal(lse, lw)
    rest = out.clone()
    rest[:, 1:2, 1:5] = 3.0
    assert torch.all(rest == 3.0)


def test_the_binding_refuses_what_does_not_fit(sa):
    c = Case([70, 64], 4, 2, 64, "bf16", seed=22)
    q, t, l = c.q.cuda(), dev(c.table), dev(c.lens)
    ok = dict(q=q, k_cache=c.kc, v_cache=c.vc, page_table=t, seq_lens=l)
    sa.sa_attn_decode(**ok)
    rp, ci = dev([0, 1, 2, 3, 4]), dev([0, 0, 0, 0])
    for bad in (dict(q=q.float()), dict(q=q[:1]), dict(q=q[:, 0]), dict(seq_lens=l[:1]),
                dict(seq_lens=l.long()), dict(seq_lens=l.cpu()), dict(page_table=t.long()),
                dict(page_table=t[0]), dict(page_table=t.t().contiguous().t()),
                dict(k_cache=c.kc[:1]), dict(k_cache=c.kc.transpose(2, 3)),
                dict(v_cache=c.vc.float()), dict(q=q.transpose(2, 3).contiguous().transpose(2, 3)),
                dict(row_ptr=rp), dict(row_ptr=rp[:4], col_idx=ci), dict(row_ptr=rp, col_idx=ci.long()),
                dict(o=q.float()), dict(o=q[:, :, :2]), dict(lse=torch.zeros(3, device="cuda")),
                dict(k_scale=torch.ones(3, device="cuda")), dict(dev_status=l.long()),
                dict(scale="x"), dict(workspace=torch.zeros((4, 4), device="cuda").t()[1:])):
        with pytest.raises(ValueError):
            sa.sa_attn_decode(**{**ok, **bad})
    for bad, code in ((dict(k_scale=torch.ones(2, device="cuda")), 1),       # scales of a bf16 cache
                      (dict(q=q.expand(2, 1, 4, 64)[:, :, :3]), 1),          # 3 heads on 2
                      (dict(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")), 3)):
        with pytest.raises(sa.SaError) as e:
            sa.sa_attn_decode(**{**ok, **bad})
        assert e.value.code == code
    sa.sa_attn_decode(**ok)
    torch.cuda.synchronize()


def test_without_lse_and_with_a_dirty_workspace(sa):
    c = Case([5000, 64], 8, 1, 128, "bf16", seed=17)
    want, _ = c.run(sa)
    p = sa.make_cache_params(dev(c.table), q=c.q.cuda(), k_cache=c.kc, v_cache=c.vc)
    n = sa.sa_attn_decode_workspace_bytes(p)
    guard = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    o, lse = c.run(sa, want_lse=False, workspace=guard[:n])
    assert lse is None and torch.equal(o, want)
    assert torch.all(guard[n:] == 0xA5)


def test_calls_repeat_bit_for_bit_captured_and_on_other_streams(sa):
    c = Case([9000, 64, 300, 0], 14, 2, 128, "bf16", seed=18)
    want, lw = c.run(sa)
    g = lambda t: t.cuda()
    q, t, l = g(c.q), dev(c.table), dev(c.lens)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        o, lse = sa.sa_attn_decode(q, c.kc, c.vc, t, l)
    for _ in range(3):
        o.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(lse, lw)
    # the lengths are read when the graph runs
    l.copy_(dev([64, 64, 64, 64]))
    graph.replay()
    torch.cuda.synchronize()
    c.lens = [64, 64, 64, 0]
    l.copy_(dev(c.lens))
    graph.replay()
    torch.cuda.synchronize()
    c.check(o, lse)
    # two calls at once, each with its own workspace
    l.copy_(dev([9000, 64, 300, 0]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [sa.sa_attn_decode(q, c.kc, c.vc, t, l, stream=s) for s in streams for _ in range(2)]
    torch.cuda.synchronize()
    for o, lse in got:
        assert torch.equal(o, want) and torch.equal(lse, lw)
