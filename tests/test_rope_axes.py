"""Rotary positions with several axes, in sa_qk_prologue and sa_cache_append, against the
fp64 definition. Bounds as those of one axis: fp32 arithmetic is off by at most 2e-6 of the
terms a value is summed from, and it is rounded once (half a bf16 step is 2^-8 of the
value, half an e4m3 step 2^-4 of it or 2^-10 of a scale)."""

import numpy as np
import pytest
import torch

from cache_helpers import PAGE, dev, new_cache, page_table, raw, status, values
from helpers import lib
from oracle.cache_oracle import places, turn_ref
from test_cache_append import check_stored

pytestmark = pytest.mark.gpu
FP32 = 2e-6


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return lib()


def axis_list(axes, D):
    """The axis of each pair, -1 where none turns it."""
    if len(axes) == D // 2:
        return list(axes)
    of = [a for a, n in enumerate(axes) for _ in range(n)]
    return of + [-1] * (D // 2 - len(of))


def angles(cos, sin, pos, of):
    """cos, sin [..., D/2] of positions [..., n_axes]."""
    of = np.array(of)
    row = np.clip(pos[..., np.maximum(of, 0)], 0, cos.shape[0] - 1)
    i = np.arange(len(of))
    return np.where(of < 0, 1.0, cos[row, i]), np.where(of < 0, 0.0, sin[row, i])


def some_tables(rows, D, gen):
    return torch.randn((rows, D // 2), generator=gen), torch.randn((rows, D // 2), generator=gen)


AXES = [((16, 8, 8), 64), ((16, 24, 24), 128), ((5, 9, 3), 64), ((1, 2, 61), 128), ((64,), 128),
        ([i % 3 for i in range(32)], 64), ([(i % 4) - 1 for i in range(64)], 128), ((0, 3, 0, 7), 64),
        ((8,) * 8, 128)]


def n_axes(axes, D):
    return max(axes) + 1 if len(axes) == D // 2 else len(axes)


@pytest.mark.parametrize("B,S,H", [(1, 1, 1), (1, 64, 3), (2, 65, 8), (1, 200, 9), (3, 127, 2)])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("axes,D", AXES, ids=str)
def test_prologue(sa, axes, D, norm, B, S, H):
    gen = torch.Generator().manual_seed(S + D)
    q, k = (torch.randn((B, S, H, D), generator=gen).to(torch.bfloat16) for _ in range(2))
    g = [1 + 0.1 * torch.randn(D, generator=gen) for _ in range(2)] if norm else [None, None]
    cos, sin = some_tables(50, D, gen)
    n = n_axes(axes, D)
    pos = torch.randint(0, 50, (B, S, n), generator=gen, dtype=torch.int32)
    c = lambda t: None if t is None else t.cuda()
    st = status()
    args = dict(gamma_q=c(g[0]), gamma_k=c(g[1]), cos=c(cos), sin=c(sin), qk_norm=norm,
                positions=c(pos), axes=axes, dev_status=st)
    qo, ko, ws = sa.sa_qk_prologue(c(q), c(k), **args)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    co, si = angles(cos.double().numpy(), sin.double().numpy(), pos.numpy(), axis_list(axes, D))
    for x, gamma, got in ((q, g[0], qo), (k, g[1], ko)):
        y, mag = turn_ref(x.double().numpy(), gamma.double().numpy() if norm else False, 1e-6,
                          co[:, :, None], si[:, :, None], "interleaved")
        check_stored(got.cpu().double().numpy(), y, mag, "bf16", None)
    # the block means it leaves are those of its outputs: the routes agree
    got = sa.sa_route_pooled(qo, ws, prefix_len=min(S, 3), tau=1.0)
    exp = sa.sa_route(qo, ko, min(S, 3), 1.0)
    assert torch.equal(got[0], exp[0])
    nnz = int(exp[0][-1])
    assert torch.equal(got[1][:nnz], exp[1][:nnz])
    # in place
    q2, k2 = c(q).clone(), c(k).clone()
    sa.sa_qk_prologue(q2, k2, q_out=q2, k_out=k2, **args)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)


def test_one_axis_by_place_is_the_plain_prologue(sa):
    """The same formula; the kernels may order their products differently, so both are held
    to the bound, and where no rounding is near the two agree to half a step."""
    gen = torch.Generator().manual_seed(1)
    q, k = (torch.randn((2, 100, 4, 128), generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    cos, sin = (t.cuda() for t in some_tables(100, 128, gen))
    plain = sa.sa_qk_prologue(q, k, cos=cos, sin=sin)
    for kw in (dict(axes=(64,)), dict(axes=[0] * 64),
               dict(positions=torch.arange(100, dtype=torch.int32, device="cuda")[None].expand(2, 100))):
        got = sa.sa_qk_prologue(q, k, cos=cos, sin=sin, **kw)
        for a, b in zip(got[:2], plain[:2]):
            off = (a.float() - b.float()).abs()
            assert bool((off <= 2.0 ** -7 * b.float().abs() + 1e-5).all())


def test_strided_positions_and_queries(sa):
    gen = torch.Generator().manual_seed(2)
    wide = torch.randn((2, 70, 5, 96), generator=gen).to(torch.bfloat16).cuda()
    q, k = wide[:, :, :2, 16:80], wide[:, :, 2:4, 16:80]
    cos, sin = (t.cuda() for t in some_tables(30, 64, gen))
    pos = torch.randint(0, 30, (1, 70, 7), generator=gen, dtype=torch.int32).cuda()
    view = pos[:, :, 2:5].expand(2, 70, 3)
    one = sa.sa_qk_prologue(q, k, cos=cos, sin=sin, positions=view, axes=(10, 10, 10))
    two = sa.sa_qk_prologue(q.contiguous(), k.contiguous(), cos=cos, sin=sin,
                            positions=view.contiguous(), axes=(10, 10, 10))
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


def test_positions_outside_the_tables_count_as_the_nearest(sa):
    gen = torch.Generator().manual_seed(3)
    q, k = (torch.randn((1, 5, 2, 64), generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    v = k.clone()
    cos, sin = (t.cuda() for t in some_tables(10, 64, gen))
    pos = dev([[[0, 3], [-7, 2], [4, 10], [9, 1 << 30], [1, 1]]])
    near = dev([[[0, 3], [0, 2], [4, 9], [9, 9], [1, 1]]])
    st = status()
    a = sa.sa_qk_prologue(q, k, cos=cos, sin=sin, positions=pos, axes=(16, 16), dev_status=st)
    assert int(st.item()) == sa.SA_DEV_CAPACITY
    b = sa.sa_qk_prologue(q, k, cos=cos, sin=sin, positions=near, axes=(16, 16))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    got = []
    for p in (pos, near):
        kc, vc = (torch.zeros((3, 2, PAGE, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        st = status()
        out = torch.zeros(1, dtype=torch.int32, device="cuda")
        qo = sa.sa_cache_append(k, v, kc, vc, dev([[1, 0]]), dev([62]), q=q, cos=cos, sin=sin, positions=p,
                                axes=(16, 16), lens_out=out, dev_status=st)
        got.append((qo, kc, vc))
        assert out.tolist() == [67]            # no token is left out for its position
        assert int(st.item()) == (sa.SA_DEV_CAPACITY if p is pos else 0)
    assert all(torch.equal(x, y) for x, y in zip(*got))


def same(a, b):
    """Equal values; a NaN is one whatever its bits."""
    return np.array_equal(a.float().cpu().numpy(), b.float().cpu().numpy(), equal_nan=True)


def test_pairs_that_stay_keep_their_values(sa):
    """Infinities and NaN beside them, or in them, are not their affair; without the norm
    they come out as they went in."""
    D = 64
    gen = torch.Generator().manual_seed(4)
    x = torch.randn((1, 70, 2, D), generator=gen).to(torch.bfloat16)
    x[0, 3, 0, 40] = float("inf")
    x[0, 4, 1, 50] = float("nan")
    x[0, 5, 0, 2] = float("inf")
    x = x.cuda()
    cos, sin = (t.cuda() for t in some_tables(70, D, gen))
    for rope, stay in (("interleaved", [d for d in range(D) if d // 2 >= 12]),
                       ("half", [d for d in range(D) if d % 32 >= 12])):
        if rope == "interleaved":
            q, k, _ = sa.sa_qk_prologue(x, x, cos=cos, sin=sin, qk_norm=False, axes=(5, 7))
            for y in (q, k):
                assert same(y[..., stay], x[..., stay])
        kc, vc = (torch.zeros((2, 2, PAGE, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        qo = sa.sa_cache_append(x, x, kc, vc, dev([[0, 1]]), dev([0]), q=x, cos=cos, sin=sin, rope=rope, axes=(5, 7))
        got = kc.permute(0, 2, 1, 3).reshape(128, 2, D)[:70]
        assert same(qo[..., stay], x[..., stay])
        assert same(got[..., stay], x[0][..., stay])


@pytest.mark.parametrize("rope", ["interleaved", "half"])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("axes,D", AXES, ids=str)
@pytest.mark.parametrize("B,S,H,Hkv,lens,new", [
    (3, 1, 8, 2, [0, 63, 300], None), (2, 2, 5, 5, [62, 10], [2, 1]), (4, 70, 14, 2, [0, 1, 64, 100], [70, 0, 33, 64])])
def test_append(sa, B, S, H, Hkv, lens, new, axes, D, norm, fmt, rope):
    gen = torch.Generator().manual_seed(B + S + D)
    after = [n + (S if new is None else new[b]) for b, n in enumerate(lens)]
    max_pages = max((a + PAGE - 1) // PAGE for a in after)
    n_pages = B * max_pages + 2
    table = page_table(after, max_pages, n_pages, gen)
    r = lambda *s: torch.randn(s, generator=gen)
    q, k, v = (r(B, S, h, D).to(torch.bfloat16) for h in (H, Hkv, Hkv))
    g = [1 + 0.1 * r(D), 1 + 0.1 * r(D)] if norm else [None, None]
    cos, sin = some_tables(40, D, gen)
    n = n_axes(axes, D)
    pos = torch.randint(0, 40, (B, S, n), generator=gen, dtype=torch.int32)
    if new is not None:                        # what does not count is not looked at
        for b in range(B):
            pos[b, new[b]:] = -5
    kc, _ = new_cache(n_pages, Hkv, D, fmt, fill=1.0, gen=gen)
    vc, _ = new_cache(n_pages, Hkv, D, fmt, fill=1.0, gen=gen)
    ks = vs = None
    if fmt == "fp8":
        ks, vs = 0.01 + 0.03 * torch.rand(Hkv, generator=gen), 0.01 + 0.03 * torch.rand(Hkv, generator=gen)
    before = raw(kc).copy(), raw(vc).copy()
    sums = r(n_pages, Hkv, D).cuda()
    s0 = sums.cpu().double().numpy()
    c = lambda t: None if t is None else t.cuda()
    st, out = status(), torch.zeros(B, dtype=torch.int32, device="cuda")
    qo = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    sa.sa_cache_append(c(k), c(v), kc, vc, dev(table), dev(lens), q=c(q), q_out=qo, new_lens=dev(new),
                       qk_norm=norm, gamma_q=c(g[0]), gamma_k=c(g[1]), cos=c(cos), sin=c(sin), rope=rope,
                       positions=c(pos), axes=axes, k_scale=c(ks), v_scale=c(vs), k_sum=sums, lens_out=out,
                       dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and out.tolist() == after
    of = axis_list(axes, D)
    co, si = angles(cos.double().numpy(), sin.double().numpy(), pos.numpy(), of)
    gam = lambda t: t.double().numpy() if norm else False
    yk, mk = turn_ref(k.double().numpy(), gam(g[1]), 1e-6, co[:, :, None], si[:, :, None], rope)
    yq, mq = turn_ref(q.double().numpy(), gam(g[0]), 1e-6, co[:, :, None], si[:, :, None], rope)
    gk, gv = values(kc, ks), values(vc, vs)
    sc = [np.ones((Hkv, 1)) if t is None else t.double().numpy()[:, None] for t in (ks, vs)]
    got_q = qo.cpu().double().numpy()
    touched, total, mags = set(), s0.copy(), np.abs(s0)
    for b, s, t in places(lens, new, S, max_pages):
        p = table[b, t // PAGE]
        check_stored(gk[p, :, t % PAGE], yk[b, s], mk[b, s], fmt, sc[0])
        check_stored(gv[p, :, t % PAGE], v[b, s].double().numpy(), 0 * mk[b, s], fmt, sc[1])
        check_stored(got_q[b, s], yq[b, s], mq[b, s], "bf16", None)
        touched.add((p, t % PAGE))
        if t % PAGE == 0:
            total[p], mags[p] = 0, 0
        total[p] += yk[b, s]
        mags[p] += np.abs(yk[b, s]) + mk[b, s]
    assert np.all(np.abs(sums.cpu().double().numpy() - total) <= (65 * 2.0 ** -24 + FP32) * mags)
    keep = np.ones((n_pages, PAGE), dtype=bool)
    for p, s in touched:
        keep[p, s] = False
    for t, b4 in ((kc, before[0]), (vc, before[1])):
        x, y = (z.reshape(n_pages, Hkv, PAGE, -1).swapaxes(1, 2) for z in (raw(t), b4))
        assert np.array_equal(x[keep], y[keep])
    idle = np.ones((B, S), dtype=bool)
    for b, s, _ in places(lens, new, S, max_pages):
        idle[b, s] = False
    assert np.all(got_q[idle] == 9.0)


def test_by_place_is_the_plain_append(sa):
    """One axis without positions: the rows by place, bit for bit."""
    gen = torch.Generator().manual_seed(8)
    for S, rope in ((1, "half"), (100, "interleaved")):
        k, v, q = (torch.randn((2, S, h, 128), generator=gen).to(torch.bfloat16).cuda() for h in (2, 2, 8))
        cos, sin = (t.cuda() for t in some_tables(400, 128, gen))
        table, lens = dev([[0, 1, 2], [3, 4, 5]]), dev([50, 3])
        got = []
        for kw in (dict(), dict(axes=(64,)), dict(positions=(lens[:, None] + torch.arange(S, device="cuda")).int())):
            kc, vc = (torch.zeros((6, 2, PAGE, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
            ksum = torch.zeros((6, 2, 128), device="cuda")
            qo = sa.sa_cache_append(k, v, kc, vc, table, lens, q=q, qk_norm=True, cos=cos, sin=sin, rope=rope,
                                    k_sum=ksum, **kw)
            got.append((qo, kc, vc, ksum))
        for other in got[1:]:
            assert all(torch.equal(x, y) for x, y in zip(got[0], other))


def test_captured_and_refused(sa):
    gen = torch.Generator().manual_seed(9)
    x = torch.randn((2, 3, 2, 64), generator=gen).to(torch.bfloat16).cuda()
    cos, sin = (t.cuda() for t in some_tables(20, 64, gen))
    pos = torch.zeros((2, 3, 3), dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros((4, 2, PAGE, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table, lens, qo = dev([[0, 1], [2, 3]]), dev([5, 6]), torch.zeros_like(x)
    call = lambda **kw: sa.sa_cache_append(x, x, kc, vc, table, lens, q=x, q_out=qo,
                                           **{**dict(cos=cos, sin=sin, positions=pos, axes=(8, 8, 8)), **kw})
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    torch.cuda.synchronize()
    pos.copy_(torch.randint(0, 20, pos.shape, generator=gen, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    replayed = qo.clone()
    call()
    assert torch.equal(replayed, qo)
    for kw in (dict(positions=pos[:, :2]), dict(positions=pos.long()), dict(axes=(8, 8)), dict(axes=(30, 8, 8)),
               dict(axes=None), dict(axes=[7] * 32), dict(positions=pos.cpu()), dict(cos=None, sin=None),
               dict(axes=(-1, 8, 8)), dict(positions=pos.transpose(0, 2))):
        with pytest.raises(ValueError):
            call(**kw)
        if kw != dict(cos=None, sin=None) and "positions" not in kw:
            with pytest.raises(ValueError):
                sa.sa_qk_prologue(x, x, **{**dict(cos=cos, sin=sin, positions=pos, axes=(8, 8, 8)), **kw})
    with pytest.raises(ValueError):
        sa.sa_qk_prologue(x, x, positions=pos, axes=(8, 8, 8))
    with pytest.raises(ValueError):
        sa.sa_qk_prologue(x, x, qk_norm=False)
    with pytest.raises(sa.SaError):
        g = torch.ones(64, device="cuda")
        sa.sa_qk_prologue(x, x, g, g, cos=cos, sin=sin, positions=pos, axes=(8, 8, 8), qk_norm=False)
    torch.cuda.synchronize()
