"""The calls on drafted tokens, pages and axes on the host, without a GPU: sizes, refusals
of the C ABI before anything is launched, of the binding, and the oracle by hand."""

import ctypes

import numpy as np
import pytest
import torch

from helpers import lib
from oracle.tree_oracle import (accept_ref, ancestors_ref, compact_ref, fork_ref, path_ref, resize_ref,
                                tree_ref)
from test_cache_host import A, CAPACITY, INVALID, UNSUPPORTED, params

FAR = 1 << 30
P = lambda x: ctypes.c_void_p(x)


@pytest.fixture(scope="module")
def sa():
    return lib()


def tree(sa, p, **kw):
    a = dict(q=A, kc=A, vc=A, k_scale=None, v_scale=None, table=A, lens=A, new=None, parents=None, stride=0,
             row_ptr=None, col_idx=None, cap=0, o=P(FAR), lse=None, ws=A, n=1 << 40)
    a.update(kw)
    return sa.load_library().sa_attn_tree(ctypes.byref(p), *a.values(), None, None)


def accept(sa, p, **kw):
    a = dict(kc=A, vc=A, k_scale=None, k_sum=None, table=A, lens=A, path=A, stride=p.S, path_lens=A, lens_out=None)
    a.update(kw)
    return sa.load_library().sa_cache_accept(ctypes.byref(p), *a.values(), None, None)


def copy(sa, p, **kw):
    a = dict(kc=A, vc=A, k_sum=None, moves=A, cap=5, n=None)
    a.update(kw)
    return sa.load_library().sa_cache_copy(ctypes.byref(p), *a.values(), None, None)


def axes(sa, D=128, n=3, rows=10, of=None, **kw):
    x = sa.sa_rope_axes()
    x.positions, x.n_axes, x.rows = 4096, n, rows
    x.pos_stride[:] = (30, 3)
    x.axis_of[: D // 2] = of or [i % n for i in range(D // 2)]
    for k, v in kw.items():
        setattr(x, k, v)
    return x


def append_axes(sa, p, rope, **kw):
    a = dict(k=A, v=A, q=A, q_out=A, gamma_q=None, gamma_k=None, cos=A, sin=A, x=ctypes.byref(rope), kc=A, vc=A,
             k_scale=None, v_scale=None, k_sum=None, table=A, lens=A, new=None, lens_out=None)
    a.update(kw)
    return sa.load_library().sa_cache_append_axes(ctypes.byref(p), *a.values(), None, None)


def prologue_axes(sa, rope, **kw):
    p = sa.sa_params()
    sa.load_library().sa_params_init(ctypes.byref(p), 2, 10, 4, 128, 0, 1.0)
    a = dict(q=A, k=A, norm=1, gamma_q=None, gamma_k=None, eps=1e-6, cos=A, sin=A, x=ctypes.byref(rope), q_out=A,
             k_out=A, ws=A, n=1 << 40)
    a.update(kw)
    return sa.load_library().sa_qk_prologue_axes(ctypes.byref(p), *a.values(), None, None)


def test_tree_sizes_and_refusals(sa):
    p = params(sa, S=5)
    size = lambda **kw: sa.load_library().sa_attn_tree_workspace_bytes(ctypes.byref(params(sa, **kw)))
    assert size(S=1) > 0 and size(S=64) >= size(S=1) and size(S=65) == 0 and size(S=4, D=96) == 0
    assert tree(sa, params(sa, S=65)) == UNSUPPORTED
    for kw in (dict(q=None), dict(kc=None), dict(o=None), dict(ws=None), dict(table=None), dict(lens=None),
               dict(row_ptr=A), dict(col_idx=A), dict(cap=-1), dict(k_scale=A), dict(q=P(4104)), dict(o=A),
               dict(parents=A, stride=4), dict(parents=A, stride=-5), dict(ws=P(4097))):
        assert tree(sa, p, **kw) == INVALID, kw
    assert tree(sa, p, n=100) == CAPACITY
    for field, value, code in (("B", 0, INVALID), ("D", 32, UNSUPPORTED), ("H", 7, INVALID),
                               ("softmax_scale", -1.0, INVALID), ("table_stride", 1, INVALID)):
        assert tree(sa, params(sa, S=5, **{field: value})) == code
    # the list of pages in 31 bits
    assert tree(sa, params(sa, S=64, B=60000, max_pages=1 << 20, table_stride=1 << 20)) == UNSUPPORTED


def test_accept_refusals(sa):
    p = params(sa, S=5)
    assert accept(sa, params(sa, S=65)) == UNSUPPORTED
    for kw in (dict(kc=None), dict(vc=None), dict(path=None), dict(path_lens=None), dict(table=None),
               dict(lens=None), dict(k_sum=P(4100)), dict(stride=4), dict(lens_out=A), dict(k_scale=A)):
        assert accept(sa, p, **kw) == INVALID, kw
    assert accept(sa, p, lens=P(FAR), path_lens=P(2 * FAR), lens_out=P(2 * FAR + 4)) == INVALID


def test_copy_refusals(sa):
    p = params(sa)
    for kw in (dict(kc=None), dict(vc=None), dict(moves=None), dict(cap=0), dict(k_sum=P(4100)), dict(kc=P(4104))):
        assert copy(sa, p, **kw) == INVALID, kw
    assert copy(sa, p, cap=1 << 31) == UNSUPPORTED


def test_pages_refusals(sa):
    L = sa.load_library()
    n = L.sa_pages_workspace_bytes(100, 7)
    assert n > 0 and L.sa_pages_workspace_bytes(0, 7) == 0 and L.sa_pages_workspace_bytes(100, 0) == 0
    assert L.sa_pages_workspace_bytes(1 << 25, 1) == 0 and L.sa_pages_workspace_bytes(5, 16385) == 0
    assert n >= 4 * (2 * 7 + 3 * 100)

    def fork(**kw):
        a = dict(n_pages=100, max_pages=5, B=7, N=6, table=A, stride=5, lens=A, refs=A, src=A, out=P(FAR), out_stride=5,
                 lens_out=P(FAR), refs_out=A, moves=A, n_moves=A, ws=A, n=n)
        a.update(kw)
        return L.sa_pages_fork(*a.values(), None, None)

    for kw in (dict(n_pages=0), dict(max_pages=0), dict(B=0), dict(N=0), dict(table=None), dict(stride=4),
               dict(out_stride=4), dict(lens=None), dict(refs=None), dict(src=None), dict(out=None),
               dict(lens_out=None), dict(refs_out=None), dict(moves=None), dict(n_moves=None), dict(ws=None),
               dict(ws=P(4100)), dict(out=A), dict(out=P(4096 + 34 * 4)), dict(lens_out=P(4096 + 24)),
               dict(refs_out=P(4100))):
        assert fork(**kw) == INVALID, kw
    assert fork(n=n - 1) == CAPACITY
    assert fork(N=16385) == UNSUPPORTED and fork(n_pages=1 << 25) == UNSUPPORTED

    def resize(**kw):
        a = dict(n_pages=100, max_pages=5, B=7, table=A, stride=5, refs=A, lens=A, more_lens=None, more=1, ws=A, n=n)
        a.update(kw)
        return L.sa_pages_resize(*a.values(), None, None)

    for kw in (dict(n_pages=0), dict(B=0), dict(table=None), dict(stride=0), dict(refs=None), dict(lens=None),
               dict(ws=None)):
        assert resize(**kw) == INVALID, kw
    assert resize(n=8) == CAPACITY and resize(max_pages=1 << 25, stride=1 << 25) == UNSUPPORTED

    def compact(**kw):
        a = dict(n_pages=100, max_pages=5, B=7, table=A, stride=5, refs=A, out=A, out_stride=5, refs_out=A, moves=A,
                 n_moves=A, n_used=A, ws=A, n=n)
        a.update(kw)
        return L.sa_pages_compact(*a.values(), None, None)

    for kw in (dict(n_pages=0), dict(B=-1), dict(B=0), dict(table=None), dict(out=None), dict(refs=None),
               dict(refs_out=None), dict(moves=None), dict(n_moves=None), dict(n_used=None), dict(out_stride=6),
               dict(out=P(4100)), dict(refs_out=P(4092)), dict(ws=P(4100))):
        assert compact(**kw) == INVALID, kw
    assert compact(n=100) == CAPACITY


def test_axes_refusals(sa):
    p = params(sa, S=10)
    bad = [dict(n=0, of=[0] * 64), dict(n=9), dict(rows=0), dict(of=[3] * 64), dict(of=[0] * 63 + [254]),
           dict(positions=4097), dict(pos_stride=(ctypes.c_int64 * 2)(-1, 3)),
           dict(pos_stride=(ctypes.c_int64 * 2)(30, -3))]
    for kw in bad:
        x = axes(sa, **kw)
        assert append_axes(sa, p, x) == INVALID and prologue_axes(sa, x) == INVALID, kw
    x = axes(sa)
    for kw in (dict(x=None), dict(cos=None), dict(sin=None), dict(gamma_q=A), dict(cos=P(4100))):
        assert append_axes(sa, p, x, **kw) == INVALID, kw
    for kw in (dict(x=None), dict(cos=None), dict(sin=None), dict(norm=2), dict(norm=0, gamma_q=A), dict(eps=-1.0),
               dict(gamma_k=P(4100)), dict(q=None), dict(k_out=None)):
        assert prologue_axes(sa, x, **kw) == INVALID, kw
    assert prologue_axes(sa, x, n=16) == CAPACITY
    assert ctypes.sizeof(sa.sa_rope_axes) == 8 + 16 + 8 + 64


def test_axes_of_the_binding(sa):
    of, n = sa._axis_bytes((2, 0, 3), 3, 64)
    assert n == 3 and list(of) == [0, 0, 2, 2, 2] + [255] * 27
    of, n = sa._axis_bytes(tuple([1, -1] * 16), 2, 64)
    assert n == 2 and list(of) == [1, 255] * 16
    assert sa._axis_bytes((32,), None, 64) == (bytes(32), 1)
    for args in (((2, 3), 3, 64), ((20, 20), 2, 64), ((1,) * 9, 9, 64), (tuple([2] * 32), 2, 64), ((), None, 64),
                 (tuple([-2] * 32), 3, 64)):
        with pytest.raises(ValueError):
            sa._axis_bytes(*args)


def test_status_bit_decodes(sa):
    L = sa.load_library()
    assert L.sa_dev_status_decode(sa.SA_DEV_BAD_TREE) == INVALID


def test_the_binding_refuses_host_tensors(sa):
    z = torch.zeros((2, 2, 64, 64), dtype=torch.bfloat16)
    i, n = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: sa.sa_attn_tree(z[:1, :1], z, z, i, n), lambda: sa.sa_cache_accept(z, z, i, n, i, n),
                 lambda: sa.sa_cache_copy(z, z, i), lambda: sa.sa_pages_fork(i, n, n, n),
                 lambda: sa.sa_pages_resize(i, n, n), lambda: sa.sa_pages_compact(i, n),
                 lambda: sa.sa_pages_compact(i, None), lambda: sa.sa_attn_tree(None, z, z, i, n)):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------- the oracle --

def test_oracle_ancestors():
    seen = ancestors_ref([-1, 0, 0, 2, 9], 5)
    assert [np.flatnonzero(r).tolist() for r in seen] == [[0], [0, 1], [0, 2], [0, 2, 3], [4]]
    assert np.array_equal(ancestors_ref(None, 4), np.tril(np.ones((4, 4), dtype=bool)))


def test_oracle_tree_of_a_chain_is_causal_attention():
    rng = np.random.default_rng(0)
    k, v, q = rng.standard_normal((3, 1, 64, 8)), rng.standard_normal((3, 1, 64, 8)), rng.standard_normal((1, 4, 2, 8))
    table = np.array([[2, 0]])
    o, lse, _, written = tree_ref(q, k, v, table, [62], None, None, 0.5)
    kk, vv = (np.concatenate([x[2, 0], x[0, 0]]) for x in (k, v))
    for s in range(4):
        x = 0.5 * q[0, s] @ kk[: 63 + s].T
        w = np.exp(x) / np.exp(x).sum(-1, keepdims=True)
        assert np.allclose(o[0, s], w @ vv[: 63 + s]) and np.allclose(lse[0, :, s], np.log(np.exp(x).sum(-1)))
    assert written.all()


def test_oracle_path_and_accept():
    assert path_ref([0, 2, 2, 5], 4, 0, 9) == [0, 2] and path_ref([1, 3, 63, 64], 4, 0, 9) == [1, 3, 63]
    assert path_ref([0, 1, 2], 3, 62, 1) == [0, 1]
    k = np.arange(2 * 64.0).reshape(2, 1, 64, 1).copy()
    v, s = -k, np.zeros((2, 1, 1))
    ends = accept_ref(k, v, s, np.array([[1, 0]]), [63], np.array([[1, 4]]), [2])
    assert ends == [65] and k[1, 0, 63, 0] == 0.0 and k[0, 0, 0, 0] == 3.0 and v[0, 0, 0, 0] == -3.0
    assert s[1, 0, 0] == sum(range(64, 127)) and s[0, 0, 0] == 3.0


def test_oracle_pages_by_hand():
    table, refs = np.array([[3, 5], [0, -1]]), np.array([1, 0, 0, 1, 0, 1, 2])
    t, n, r, moves, short = fork_ref(table, [100, 10], refs, [0, 0, -1, 1])
    assert t.tolist() == [[3, 5], [3, 1], [-1, -1], [0, -1]] and n == [100, 100, 0, 10] and moves == [(5, 1)]
    assert r.tolist() == [1, 1, 0, 2, 0, 1, 2] and not short
    t, r, short = resize_ref(table, refs, [64, 70])
    assert t.tolist() == [[3, -1], [0, 1]] and r.tolist() == [1, 1, 0, 1, 0, 0, 2] and not short
    t, r, moves, used = compact_ref(table, refs)
    assert used == 4 and moves == [(5, 1), (6, 2)] and t.tolist() == [[3, 1], [0, -1]]
    assert r.tolist() == [1, 1, 2, 1, 0, 0, 0]
