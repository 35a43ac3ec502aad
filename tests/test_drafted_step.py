"""Speculative decoding as it is used: drafts are appended by their depth, attended as a
tree, the accepted path kept, sequences forked and given pages, the pool compacted. Every
step is held against the sequences as they would stand had their tokens come one by one."""

import numpy as np
import pytest
import torch

from cache_helpers import PAGE, dev, status, values
from helpers import lib
from oracle.cache_oracle import decode_ref
from oracle.tree_oracle import ancestors_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return lib()


@pytest.mark.parametrize("fmt,rope", [("bf16", "interleaved"), ("fp8", "half")])
def test_a_loop_of_drafts(sa, fmt, rope):
    B, H, Hkv, D, S, max_pages, n_pages = 3, 8, 2, 64, 9, 6, 40
    rng, gen = np.random.default_rng(1), torch.Generator().manual_seed(1)
    dt = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
    kc, vc = (torch.zeros((n_pages, Hkv, PAGE, D), dtype=dt, device="cuda") for _ in range(2))
    ks = vs = None
    if fmt == "fp8":
        ks, vs = torch.full((Hkv,), 0.02).cuda(), torch.full((Hkv,), 0.03).cuda()
    k_sum = torch.zeros((n_pages, Hkv, D), device="cuda")
    angle = torch.arange(500)[:, None] * 1e4 ** (-torch.arange(D // 2) / (D // 2))
    cos, sin = angle.cos().cuda(), angle.sin().cuda()
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    refs, lens = torch.zeros(n_pages, dtype=torch.int32, device="cuda"), dev([0] * B)
    st = status()
    r = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16).cuda()
    turn = dict(qk_norm=True, cos=cos, sin=sin, rope=rope, k_scale=ks, v_scale=vs, k_sum=k_sum, dev_status=st)
    # prompts
    n0 = dev([70, 5, 128])
    sa.sa_pages_resize(table, refs, lens, more_lens=n0, dev_status=st)
    kp, vp = r(B, 128, Hkv, D), r(B, 128, Hkv, D)
    now = torch.zeros_like(lens)
    sa.sa_cache_append(kp, vp, kc, vc, table, lens, new_lens=n0, lens_out=now, **turn)
    # what each sequence consists of, token by token (before norm and rotation)
    history = [[(kp[b, t], vp[b, t]) for t in range(int(n0[b]))] for b in range(B)]
    for step in range(4):
        lens = now
        new = dev(rng.integers(1, S + 1, B))
        up = np.full((B, S), -1, dtype=np.int32)
        for b in range(B):
            for s in range(1, S):
                up[b, s] = rng.integers(0, s)
        depth = np.stack([ancestors_ref(up[b], S).sum(1) - 1 for b in range(B)])
        positions = (lens[:, None] + dev(depth)).int()
        sa.sa_pages_resize(table, refs, lens, S, dev_status=st)
        k, v, q = r(B, S, Hkv, D), r(B, S, Hkv, D), r(B, S, H, D)
        after = torch.zeros_like(lens)
        qr = sa.sa_cache_append(k, v, kc, vc, table, lens, q=q, new_lens=new, positions=positions, lens_out=after,
                                **turn)
        o, lse = sa.sa_attn_tree(qr, kc, vc, table, lens, parents=dev(up), new_lens=new, k_scale=ks, v_scale=vs,
                                 dev_status=st)
        # a walk from token 0 down, as a verifier takes it
        path, m = np.full((B, S), -1, dtype=np.int32), []
        for b in range(B):
            walk = [0]
            while True:
                kids = [s for s in range(walk[-1] + 1, int(new[b])) if up[b, s] == walk[-1]]
                if not kids or rng.random() < 0.2:
                    break
                walk.append(int(rng.choice(kids)))
            path[b, :len(walk)] = walk
            m.append(len(walk))
        now = torch.zeros_like(lens)
        sa.sa_cache_accept(kc, vc, table, lens, dev(path), dev(m), k_sum=k_sum, k_scale=ks, lens_out=now,
                           dev_status=st)
        for b in range(B):
            history[b] += [(k[b, a], v[b, a]) for a in path[b, :m[b]]]
        assert now.tolist() == [len(h) for h in history]
        # the same tokens one after another into a cache of their own
        kc2, vc2 = torch.zeros_like(kc), torch.zeros_like(vc)
        sum2, l2 = torch.zeros_like(k_sum), torch.zeros_like(lens)
        most = max(len(h) for h in history)
        pad = lambda i: torch.stack([torch.stack([h[min(t, len(h) - 1)][i] for t in range(most)]) for h in history])
        own = torch.arange(B * max_pages, dtype=torch.int32, device="cuda").reshape(B, max_pages)
        sa.sa_cache_append(pad(0), pad(1), kc2, vc2, own, l2, new_lens=now, **{**turn, "k_sum": sum2})
        for b in range(B):
            for j in range(-(-len(history[b]) // PAGE)):
                live = min(PAGE, len(history[b]) - PAGE * j)
                p1, p2 = int(table[b, j]), int(own[b, j])
                for x, y in ((kc, kc2), (vc, vc2)):
                    x, y = (t.view(torch.uint8) if fmt == "fp8" else t for t in (x, y))
                    assert torch.equal(x[p1, :, :live], y[p2, :, :live])
                # sums: of stored keys where the page was touched since, of keys before rounding
                # otherwise; a rounding is at most 2^-8 (2^-4 and half a code's least step) of each
                mag = np.abs(values(kc, ks)[p1][:, :live])
                tol = (2.0 ** -8 * mag).sum(1) if fmt == "bf16" else np.maximum(2.0 ** -4 * mag, 2.0 ** -10 * 0.02).sum(1)
                off = np.abs((k_sum[p1] - sum2[p2]).cpu().double().numpy())
                assert np.all(off <= tol * 1.02 + 65 * 2.0 ** -24 * mag.sum(1) + 1e-6)
        # the last accepted token attends, over the whole cache, what it saw in its tree
        last = torch.stack([qr[b, path[b, m[b] - 1]] for b in range(B)])[:, None].contiguous()
        o1, l1 = sa.sa_attn_decode(last, kc, vc, table, now, k_scale=ks, v_scale=vs, dev_status=st)
        for b in range(B):
            a = o[b, path[b, m[b] - 1]].float()
            assert bool(((o1[b, 0].float() - a).abs() <= 2.0 ** -6 * a.abs() + 1e-3).all())
            assert torch.allclose(l1[b, :, 0], lse[b, :, path[b, m[b] - 1]], atol=1e-4)
        # beams: sequence 2 ends, the others go on
        if step == 1:
            src = [1, 0, 1]
            table, now, refs, moves, n = sa.sa_pages_fork(table, now, refs, dev(src), dev_status=st)
            sa.sa_cache_copy(kc, vc, moves, n, k_sum=k_sum, dev_status=st)
            history = [list(history[i]) for i in src]
        if step == 2:
            table, refs, moves, n, used = sa.sa_pages_compact(table, refs, dev_status=st)
            sa.sa_cache_copy(kc, vc, moves, n, k_sum=k_sum, dev_status=st)
            assert int(table.max()) < int(used.item()) == int((refs > 0).sum())
        held = torch.bincount(table[table >= 0].long(), minlength=n_pages)
        assert torch.equal(held.int(), refs)
    # routed decoding goes on from here
    q = r(B, 1, H, D)
    row_ptr, cols = sa.sa_route_pages(q, k_sum, table, now, 0, 2, dev_status=st)
    o1, _ = sa.sa_attn_decode(q, kc, vc, table, now, row_ptr=row_ptr, col_idx=cols, k_scale=ks, v_scale=vs,
                              dev_status=st)
    rp, ci = row_ptr.tolist(), cols.tolist()
    rows = [ci[rp[i]:rp[i + 1]] for i in range(B * Hkv)]
    ref, _, mag = decode_ref(q[:, 0].double().cpu().numpy(), values(kc, ks), values(vc, vs), table.cpu().numpy(),
                             now.tolist(), D ** -0.5, rows)
    off = np.abs(o1[:, 0].double().cpu().numpy() - ref)
    assert np.all(off <= 2.0 ** -8 * np.abs(ref) + 1e-3 * mag)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
