"""sa_cache_append against the fp64 definition.

Bounds, all from the arithmetic. The normed and rotated value is computed in
fp32 with an error of at most 2e-6 of the terms it is summed from (sum of
squares, a reciprocal root of 2 ulp, two products, a rotation) and is rounded
once: half a bf16 step is 2^-8 of the value, half an e4m3 step 2^-4 of it, or
2^-10 of a scale for codes below the normal range. A page's sum adds at most 64
such terms and an old sum in fp32: 65 roundings of at most 2^-24 of the sum of
the magnitudes."""

import numpy as np
import pytest
import torch

from cache_helpers import PAGE, dev, new_cache, page_table, raw, status, values
from helpers import lib
from oracle.cache_oracle import places, turn_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return lib()


FP32 = 2e-6


def check_stored(got, exact, mag, fmt, scale):
    """Stored values against exact ones, with the fp32 error FP32 * mag."""
    if fmt == "bf16":
        tol = 2.0 ** -8 * np.abs(exact) + FP32 * mag
    else:
        top = 448.0 * scale
        exact = np.clip(exact, -top, top)
        tol = np.maximum(2.0 ** -4 * np.abs(exact), 2.0 ** -10 * scale) + FP32 * mag
    assert np.all(np.abs(got - exact) <= tol * (1 + 1e-6)), \
        float(np.max(np.abs(got - exact) / np.maximum(tol, 1e-300)))


class Case:
    def __init__(self, B, S, H, Hkv, D, fmt, lens, new=None, norm=True, gamma=True, rope="interleaved",
                 sums=True, layout="page_head", scales=True, extra_pages=0, seed=0, fill=1.0,
                 rope_rows=None):
        gen = torch.Generator().manual_seed(seed)
        self.__dict__.update(B=B, S=S, H=H, Hkv=Hkv, D=D, fmt=fmt, lens=lens, new=new, norm=norm,
                             rope=rope)
        after = [n + (S if new is None else new[b]) for b, n in enumerate(lens)]
        self.max_pages = max(1, max((max(a, 0) + PAGE - 1) // PAGE for a in after)) + extra_pages
        self.n_pages = B * self.max_pages + 2
        self.table = page_table(after, self.max_pages, self.n_pages, gen)
        r = lambda *s: torch.randn(s, generator=gen)
        self.k, self.v = (r(B, S, Hkv, D).to(torch.bfloat16) for _ in range(2))
        self.q = r(B, S, H, D).to(torch.bfloat16) if H else None
        self.gq = self.gk = self.cos = self.sin = self.ks = self.vs = self.ksum = None
        if norm and gamma:
            self.gq, self.gk = 1 + 0.1 * r(D), 1 + 0.1 * r(D)
        if rope:
            rows = self.max_pages * PAGE if rope_rows is None else rope_rows
            ang = torch.arange(rows)[:, None] * 10000.0 ** (-torch.arange(D // 2) / (D // 2))
            self.cos, self.sin = ang.cos().float(), ang.sin().float()
        if fmt == "fp8" and scales:
            self.ks, self.vs = 0.005 + 0.03 * torch.rand(Hkv, generator=gen), \
                0.005 + 0.03 * torch.rand(Hkv, generator=gen)
        self.kc, self.kbuf = new_cache(self.n_pages, Hkv, D, fmt, layout, fill, gen)
        self.vc, self.vbuf = new_cache(self.n_pages, Hkv, D, fmt, layout, fill, gen)
        if sums:
            self.ksum = r(self.n_pages, Hkv, D)
        self.ksum_d = None if self.ksum is None else self.ksum.cuda()

    def run(self, sa, in_place=False, lens_out=True, **kw):
        c = lambda t: None if t is None else t.cuda()
        self.kbuf0, self.vbuf0 = self.kbuf.clone(), self.vbuf.clone()
        q = c(self.q)
        self.q_out = None if q is None else (q if in_place else torch.full_like(q, 7.0))
        self.lens_out = torch.full((self.B,), -5, dtype=torch.int32, device="cuda") if lens_out else None
        self.st = status()
        args = dict(q=q, q_out=self.q_out, new_lens=dev(self.new), qk_norm=self.norm,
                    gamma_q=c(self.gq), gamma_k=c(self.gk), eps=1e-6, cos=c(self.cos),
                    sin=c(self.sin), rope=self.rope or "interleaved", k_scale=c(self.ks),
                    v_scale=c(self.vs), k_sum=self.ksum_d, lens_out=self.lens_out,
                    dev_status=self.st)
        args.update(kw)
        sa.sa_cache_append(c(self.k), c(self.v), self.kc, self.vc, dev(self.table), dev(self.lens),
                           **args)
        torch.cuda.synchronize()
        return self

    def check(self, status=0, place=None):
        """Everything that was to be written, and nothing else."""
        place = list(places(self.lens, self.new, self.S, self.max_pages)) if place is None else place
        assert int(self.st.item()) == status
        ones = np.ones(self.Hkv)
        ks = ones if self.ks is None else self.ks.double().numpy()
        vs = ones if self.vs is None else self.vs.double().numpy()
        gk = False if not self.norm else (None if self.gk is None else self.gk.double().numpy())
        gq = False if not self.norm else (None if self.gq is None else self.gq.double().numpy())
        kval, vval = values(self.kc, self.ks), values(self.vc, self.vs)
        k64, v64 = self.k.double().numpy(), self.v.double().numpy()
        sums = {}
        for b, s, t in place:
            c = sn = None
            if self.cos is not None:
                c, sn = self.cos[t].double().numpy(), self.sin[t].double().numpy()
            y, mag = turn_ref(k64[b, s], gk, 1e-6, c, sn, self.rope)
            page, slot = self.table[b, t // PAGE], t % PAGE
            check_stored(kval[page, :, slot], y, mag, self.fmt, ks[:, None])
            check_stored(vval[page, :, slot], v64[b, s], np.abs(v64[b, s]), self.fmt, vs[:, None])
            if self.fmt == "bf16":
                assert np.array_equal(vval[page, :, slot], v64[b, s])
            if page not in sums:
                old = 0.0 if slot == 0 else self.ksum[page].double().numpy() if self.ksum is not None else 0.0
                sums[page] = [np.zeros_like(y) + old, np.abs(np.zeros_like(y) + old)]
            sums[page][0] += y
            sums[page][1] += mag
            if self.q is not None:
                y, mag = turn_ref(self.q[b, s].double().numpy(), gq, 1e-6, c, sn, self.rope)
                check_stored(self.q_out[b, s].cpu().double().numpy(), y, mag, "bf16", None)
        # nothing else changed
        for buf, old, t in ((self.kbuf, self.kbuf0, self.kc), (self.vbuf, self.vbuf0, self.vc)):
            now, was = buf.clone(), old
            # put the old values back where tokens were written, through the same view
            off = t.storage_offset()
            view = torch.as_strided(now, t.shape, t.stride(), off)
            wasv = torch.as_strided(was, t.shape, t.stride(), off)
            if now.dtype != torch.bfloat16:
                view, wasv = view.view(torch.uint8), wasv.view(torch.uint8)
            for b, s, tt in place:
                page, slot = int(self.table[b, tt // PAGE]), tt % PAGE
                view[page, :, slot] = wasv[page, :, slot]
            assert np.array_equal(raw(now), raw(was))
        if self.ksum is not None:
            got = self.ksum_d.cpu().double().numpy()
            for page in range(self.n_pages):
                if page in sums:
                    total, mag = sums[page]
                    tol = (FP32 + 65 * 2.0 ** -24) * mag
                    assert np.all(np.abs(got[page] - total) <= tol), float(np.max(np.abs(got[page] - total) / tol))
                else:
                    assert np.array_equal(got[page], self.ksum[page].double().numpy())
        if self.q is not None:
            there = np.zeros((self.B, self.S), dtype=bool)
            for b, s, _ in place:
                there[b, s] = True
            rest = self.q_out.cpu()[torch.from_numpy(~there)]
            assert torch.all(rest == 7.0)


SHAPES = [
    # B, S, H, Hkv, D, fmt, lens, new
    (1, 1, 4, 2, 128, "bf16", [0], None),
    (1, 1, 1, 1, 64, "fp8", [63], None),
    (3, 1, 14, 2, 128, "fp8", [64, 0, 1023], None),
    (2, 2, 8, 8, 64, "bf16", [63, 126], None),
    (2, 63, 6, 3, 128, "bf16", [1, 64], None),
    (1, 64, 5, 1, 64, "fp8", [0], None),
    (2, 65, 7, 1, 128, "bf16", [63, 100], [65, 0]),
    (4, 130, 10, 5, 64, "fp8", [0, 5, 64, 191], [130, 1, 64, 77]),
    (1, 515, 56, 8, 128, "bf16", [951], None),
    (300, 1, 4, 2, 64, "bf16", [(37 * i) % 200 for i in range(300)], [i % 2 for i in range(300)]),
]


@pytest.mark.parametrize("rope", ["interleaved", "half", None])
@pytest.mark.parametrize("B,S,H,Hkv,D,fmt,lens,new", SHAPES)
def test_append_matches_the_definition(sa, B, S, H, Hkv, D, fmt, lens, new, rope):
    c = Case(B, S, H, Hkv, D, fmt, lens, new, rope=rope, norm=rope != "half", seed=S + B)
    c.run(sa).check()
    n = [S if new is None else new[b] for b in range(B)]
    assert c.lens_out.tolist() == [a + b for a, b in zip(lens, n)]


@pytest.mark.parametrize("layout", ["page_token", "gapped"])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_cache_layouts_and_strided_tokens(sa, layout, fmt):
    c = Case(2, 70, 6, 3, 128, fmt, [10, 64], layout=layout, rope="half", seed=3)
    c.run(sa).check()
    # the new tokens as slices of a fused projection, heads before tokens in memory
    d = Case(2, 70, 6, 3, 128, fmt, [10, 64], layout=layout, rope="half", seed=3)
    fused = torch.zeros((2, 14, 70, 128), dtype=torch.bfloat16)
    fused[:, 0:6], fused[:, 6:9], fused[:, 9:12] = (t.transpose(1, 2) for t in (d.q, d.k, d.v))
    fused = fused.cuda()
    st = status()
    out = sa.sa_cache_append(fused[:, 6:9].transpose(1, 2), fused[:, 9:12].transpose(1, 2), d.kc,
                             d.vc, dev(d.table), dev(d.lens), q=fused[:, 0:6].transpose(1, 2),
                             qk_norm=True, gamma_q=d.gq.cuda(), gamma_k=d.gk.cuda(),
                             cos=d.cos.cuda(), sin=d.sin.cuda(), rope="half",
                             k_scale=None if d.ks is None else d.ks.cuda(),
                             v_scale=None if d.vs is None else d.vs.cuda(), k_sum=d.ksum_d,
                             dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert np.array_equal(raw(c.kbuf), raw(d.kbuf)) and np.array_equal(raw(c.vbuf), raw(d.vbuf))
    assert torch.equal(c.q_out, out) and torch.equal(c.ksum_d, d.ksum_d)


def test_without_queries_sums_scales_or_weights(sa):
    Case(2, 5, 0, 2, 64, "fp8", [0, 62], sums=False, scales=False, gamma=False).run(
        sa, lens_out=False).check()
    Case(1, 1, 3, 3, 128, "bf16", [64], norm=False, rope=None, sums=False).run(sa).check()


def test_queries_in_place(sa):
    a = Case(2, 66, 6, 2, 128, "bf16", [3, 64], seed=8).run(sa)
    b = Case(2, 66, 6, 2, 128, "bf16", [3, 64], seed=8).run(sa, in_place=True)
    assert torch.equal(a.q_out, b.q_out)


def test_one_at_a_time_equals_all_at_once(sa):
    """Keys and values bit for bit; sums within the roundings of 65 terms."""
    whole = Case(1, 130, 4, 2, 128, "fp8", [30], seed=4)
    parts = Case(1, 130, 4, 2, 128, "fp8", [30], seed=4)
    whole.run(sa)
    c = lambda t: t.cuda()
    for s in range(130):
        sa.sa_cache_append(c(parts.k[:, s:s + 1]), c(parts.v[:, s:s + 1]), parts.kc, parts.vc,
                           dev(parts.table), dev([30 + s]), qk_norm=True, gamma_k=c(parts.gk),
                           cos=c(parts.cos), sin=c(parts.sin), k_scale=c(parts.ks),
                           v_scale=c(parts.vs), k_sum=parts.ksum_d)
    torch.cuda.synchronize()
    assert np.array_equal(raw(whole.kbuf), raw(parts.kbuf))
    assert np.array_equal(raw(whole.vbuf), raw(parts.vbuf))
    tol = 2 * 65 * 2.0 ** -24 * 65 * float(whole.ksum_d.abs().max())
    assert float((whole.ksum_d - parts.ksum_d).abs().max()) <= tol


def test_tokens_without_a_place_are_left_out(sa):
    # sequence 0 fills its two pages and spills, 1 is longer than its table, 2 is negative
    c = Case(3, 40, 2, 1, 64, "bf16", [100, 10, 0], seed=1)
    c.lens = [100, 500, -3]
    assert c.max_pages == 3
    c.table = c.table[:, :2].copy()
    c.max_pages = 2
    used = set(c.table.ravel().tolist())
    c.table[2] = [page for page in range(c.n_pages) if page not in used][:2]
    c.run(sa)
    c.check(status=sa.SA_DEV_CAPACITY | sa.SA_DEV_BAD_CACHE)
    assert c.lens_out.tolist() == [128, 128, 40]


def test_bad_pages_and_short_tables(sa):
    c = Case(2, 130, 2, 2, 128, "bf16", [0, 0], seed=2)
    c.table[0, 1], c.table[1, 0] = c.n_pages, -1
    place = [(b, s, t) for b, s, t in places(c.lens, None, c.S, c.max_pages)
             if (b, t // PAGE) not in ((0, 1), (1, 0))]
    c.run(sa).check(status=sa.SA_DEV_BAD_CACHE, place=place)
    # rotation tables of 100 rows: later positions find no angle
    c = Case(1, 130, 2, 2, 128, "bf16", [0], seed=2, rope_rows=100)
    place = [(b, s, t) for b, s, t in places(c.lens, None, c.S, c.max_pages) if t < 100]
    c.run(sa).check(status=sa.SA_DEV_CAPACITY, place=place)


def test_saturation_and_not_a_number(sa):
    c = Case(1, 4, 0, 1, 64, "fp8", [0], norm=False, rope=None, scales=False, sums=False)
    c.v[0, 0, 0, :4] = torch.tensor([500.0, -1e30, float("inf"), float("nan")])
    c.v[0, 1, 0, :2] = torch.tensor([2.0 ** -10, 2.0 ** -11])    # ties to even: down to 0; 2^-11: 0
    c.run(sa)
    got = values(c.vc)[c.table[0, 0], 0]
    assert got[0, 0] == 448 and got[0, 1] == -448 and got[0, 2] == 448 and np.isnan(got[0, 3])
    assert got[1, 0] == 0 and got[1, 1] == 0


def test_pages_beyond_32_bit_offsets(sa):
    """A pool of 5 GB whose last page takes the tokens."""
    n_pages, Hkv, D = 40_000, 8, 128
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    kc, vc = (torch.empty((n_pages, Hkv, PAGE, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ksum = torch.empty((n_pages, Hkv, D), device="cuda")
    gen = torch.Generator().manual_seed(1)
    k, v = (torch.randn((1, 70, Hkv, D), generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    table = dev([[n_pages - 1, n_pages - 2]])
    sa.sa_cache_append(k, v, kc, vc, table, dev([0]), k_sum=ksum)
    torch.cuda.synchronize()
    for cache, x in ((kc, k), (vc, v)):
        assert torch.equal(cache[-1].transpose(0, 1), x[0, :64])
        assert torch.equal(cache[-2, :, :6].transpose(0, 1), x[0, 64:])
    # 64 fp32 additions: at most 64 roundings of 2^-24 of the magnitudes' sum
    want, mag = k[0, :64].double().sum(0), k[0, :64].double().abs().sum(0)
    assert torch.all((ksum[-1].double() - want).abs() <= 64 * 2.0 ** -24 * mag)


def test_the_binding_refuses_what_does_not_fit(sa):
    c = Case(2, 3, 4, 2, 64, "fp8", [5, 64], seed=7)
    g = lambda t: t.cuda()
    ok = dict(k=g(c.k), v=g(c.v), k_cache=c.kc, v_cache=c.vc, page_table=dev(c.table),
              seq_lens=dev(c.lens), q=g(c.q), qk_norm=True, gamma_q=g(c.gq), cos=g(c.cos),
              sin=g(c.sin), k_scale=g(c.ks), v_scale=g(c.vs), k_sum=c.ksum_d)
    sa.sa_cache_append(**ok)
    for bad in (dict(k=ok["k"].float()), dict(k=ok["k"][:, :2]), dict(v=ok["v"][:1]),
                dict(q=ok["q"][:, :2]), dict(q=None, q_out=ok["q"]), dict(cos=None), dict(sin=None),
                dict(cos=ok["cos"][:0], sin=ok["sin"][:0]), dict(cos=ok["cos"][:, :16], sin=ok["sin"][:, :16]),
                dict(gamma_q=ok["gamma_q"][:32]), dict(k_sum=ok["k_sum"][1:]),
                dict(k_scale=ok["k_scale"].double()), dict(new_lens=dev([1, 2, 3])),
                dict(lens_out=dev([1])), dict(k_cache=c.kc.view(torch.uint8)), dict(eps=None),
                dict(rope=1.5), dict(seq_lens=ok["seq_lens"].cpu())):
        with pytest.raises((ValueError, KeyError)):
            sa.sa_cache_append(**{**ok, **bad})
    for bad in (dict(eps=-1.0), dict(rope=7), dict(qk_norm=False), dict(lens_out=ok["seq_lens"])):
        with pytest.raises(sa.SaError) as e:
            sa.sa_cache_append(**{**ok, **bad})
        assert e.value.code == 1
    torch.cuda.synchronize()


def test_captured_and_replayed_on_another_stream(sa):
    c = Case(2, 3, 4, 2, 128, "bf16", [62, 5], sums=False, seed=6)
    e = Case(2, 3, 4, 2, 128, "bf16", [62, 5], sums=False, seed=6)
    e.run(sa)
    g = lambda t: t.cuda()
    k, v, q, t, l = g(c.k), g(c.v), g(c.q), dev(c.table), dev(c.lens)
    args = dict(q=q, qk_norm=True, gamma_q=g(c.gq), gamma_k=g(c.gk), cos=g(c.cos), sin=g(c.sin))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sa.sa_cache_append(k, v, c.kc, c.vc, t, l, **args)
    assert np.all(values(c.kc) == values(torch.as_strided(e.kbuf0, e.kc.shape, e.kc.stride())))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(raw(c.kbuf), raw(e.kbuf)) and torch.equal(out, e.q_out)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        with torch.cuda.stream(torch.cuda.current_stream()):
            out = sa.sa_cache_append(k, v, c.kc, c.vc, t, l, stream=stream, **args)
        side.synchronize()
        assert torch.equal(out, e.q_out)
