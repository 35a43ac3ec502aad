"""The paged cache on the host, without a GPU: sizes, refusals of the C ABI
before anything is launched, refusals of the binding, and the oracle."""

import ctypes
import math

import numpy as np
import pytest
import torch

from helpers import lib
from oracle.cache_oracle import decode_ref, places, route_pages_ref, turn_ref

OK, INVALID, UNSUPPORTED, CAPACITY = 0, 1, 2, 3


@pytest.fixture(scope="module")
def sa():
    return lib()


def params(sa, B=2, H=8, Hkv=2, D=128, n_pages=10, max_pages=5, **kw):
    p = sa.sa_cache_params()
    sa.load_library().sa_cache_params_init(ctypes.byref(p), B, H, Hkv, D, n_pages, max_pages)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


A = ctypes.c_void_p(4096)


def append(sa, p, **kw):
    a = dict(k=A, v=A, q=A, q_out=A, gamma_q=None, gamma_k=None, cos=None, sin=None, kc=A, vc=A,
             k_scale=None, v_scale=None, k_sum=None, table=A, lens=A, new=None, lens_out=None)
    a.update(kw)
    return sa.load_library().sa_cache_append(ctypes.byref(p), *a.values(), None, None)


def route(sa, p, **kw):
    a = dict(q=A, k_sum=A, table=A, lens=A, row_ptr=A, col_idx=A, cap=100, ws=A, n=1 << 40)
    a.update(kw)
    return sa.load_library().sa_route_pages(ctypes.byref(p), *a.values(), None, None)


def decode(sa, p, **kw):
    a = dict(q=A, kc=A, vc=A, k_scale=None, v_scale=None, table=A, lens=A, row_ptr=None,
             col_idx=None, cap=0, o=A, lse=None, ws=A, n=1 << 40)
    a.update(kw)
    return sa.load_library().sa_attn_decode(ctypes.byref(p), *a.values(), None, None)


def test_init_and_sizes(sa):
    p = params(sa)
    assert (p.S, p.page, p.table_stride, p.cache_format) == (1, 64, 5, sa.SA_CACHE_BF16)
    assert list(p.kc_stride) == [2 * 64 * 128, 64 * 128, 128] and list(p.q_stride) == [1024, 1024, 128]
    L = sa.load_library()
    n = lambda **kw: L.sa_route_pages_max_nnz(ctypes.byref(params(sa, **kw)))
    assert n(page_budget=3) == 2 * 2 * 3
    assert n(page_budget=3, prefix_len=200) == 2 * 2 * 5       # 4 sink pages and the newest
    assert n(page_budget=300) == 2 * 2 * 5
    assert L.sa_route_pages_workspace_bytes(ctypes.byref(p)) > 0
    assert L.sa_attn_decode_workspace_bytes(ctypes.byref(p)) > 0
    assert ctypes.sizeof(sa.sa_cache_params) == 14 * 4 + 2 * 4 + 8 + 18 * 8


@pytest.mark.parametrize("field,value,code", [
    ("B", 0, INVALID), ("S", 0, INVALID), ("H", 9, INVALID), ("H_kv", 0, INVALID),
    ("D", 96, UNSUPPORTED), ("D", 0, INVALID), ("page", 32, INVALID), ("n_pages", 0, INVALID),
    ("max_pages", 0, INVALID), ("max_pages", 1 << 25, INVALID), ("cache_format", 2, INVALID),
    ("rope_layout", 2, INVALID), ("prefix_len", -1, INVALID), ("page_budget", -1, INVALID),
    ("qk_norm", 2, INVALID), ("rope_rows", -1, INVALID), ("eps", -1.0, INVALID),
    ("eps", float("nan"), INVALID), ("softmax_scale", float("inf"), INVALID),
    ("softmax_scale", -1.0, INVALID), ("table_stride", 4, INVALID), ("B", 65536, UNSUPPORTED),
])
def test_bad_params(sa, field, value, code):
    p = params(sa, **{field: value})
    assert append(sa, p) == code and route(sa, p) == code and decode(sa, p) == code
    L = sa.load_library()
    assert L.sa_attn_decode_workspace_bytes(ctypes.byref(p)) == 0
    assert L.sa_route_pages_workspace_bytes(ctypes.byref(p)) == 0
    assert L.sa_route_pages_max_nnz(ctypes.byref(p)) == 0


def test_one_new_token_only(sa):
    p = params(sa, S=2)
    assert route(sa, p) == UNSUPPORTED and decode(sa, p) == UNSUPPORTED


def test_append_refusals(sa):
    p = params(sa)
    odd = ctypes.c_void_p(4096 + 8)
    for name in ("k", "v", "kc", "vc", "table", "lens", "q", "q_out"):
        assert append(sa, p, **{name: None}) == INVALID, name
    for name in ("k", "v", "q", "q_out", "kc", "vc", "k_sum", "cos"):
        kw = {name: odd}
        if name == "cos":
            kw["sin"] = A
        assert append(sa, p, **kw) == INVALID, name
    assert append(sa, p, cos=A) == INVALID and append(sa, p, sin=A) == INVALID
    assert append(sa, p, gamma_k=A) == INVALID                  # weights without the norm
    assert append(sa, p, k_scale=A) == INVALID                  # scales of a bf16 cache
    assert append(sa, p, lens_out=A) == INVALID                 # seq_lens itself
    B = ctypes.c_void_p(8192)
    assert append(sa, p, lens=B, new=A, lens_out=A) == INVALID  # new_lens itself
    p.o_stride[1] = 2048                                        # in place, laid out otherwise
    p.o_stride[0] = 2048
    assert append(sa, p) == INVALID
    p = params(sa)
    for field, i in (("q_stride", 1), ("k_stride", 0), ("v_stride", 2), ("o_stride", 2),
                     ("kc_stride", 0), ("vc_stride", 2)):
        for bad in (4, 0, -8):
            p = params(sa, S=3)
            getattr(p, field)[i] = bad
            assert append(sa, p) == INVALID, (field, bad)
    p = params(sa, cache_format=1)
    p.kc_stride[2] = 136                                        # 8 codes: not 16 bytes
    assert append(sa, p) == INVALID and decode(sa, p) == INVALID


def test_route_and_decode_refusals(sa):
    p = params(sa, page_budget=3)
    for name in ("q", "k_sum", "table", "lens", "row_ptr", "col_idx", "ws"):
        assert route(sa, p, **{name: None}) == INVALID, name
    assert route(sa, p, cap=-1) == INVALID
    assert route(sa, p, ws=ctypes.c_void_p(4096 + 128)) == INVALID
    need = sa.load_library().sa_route_pages_workspace_bytes(ctypes.byref(p))
    assert route(sa, p, n=need - 1) == CAPACITY
    big = params(sa, B=60000, H=64, Hkv=64, max_pages=1 << 20)
    assert route(sa, big) == UNSUPPORTED                        # lists beyond int32
    assert route(sa, params(sa, B=1, max_pages=(1 << 20) + 1)) == UNSUPPORTED
    assert decode(sa, big) == UNSUPPORTED                       # pages beyond 31 bits
    p = params(sa)
    for name in ("q", "kc", "vc", "table", "lens", "o", "ws"):
        assert decode(sa, p, **{name: None}) == INVALID, name
    assert decode(sa, p, row_ptr=A) == INVALID and decode(sa, p, col_idx=A) == INVALID
    assert decode(sa, p, row_ptr=A, col_idx=A, cap=-1) == INVALID
    assert decode(sa, p, ws=ctypes.c_void_p(4096 + 16)) == INVALID
    need = sa.load_library().sa_attn_decode_workspace_bytes(ctypes.byref(p))
    assert decode(sa, p, n=need - 1) == CAPACITY
    assert sa.load_library().sa_dev_status_decode(sa.SA_DEV_BAD_CACHE) == INVALID


def test_decode_does_not_write_over_its_queries(sa):
    p = params(sa)
    need = sa.load_library().sa_attn_decode_workspace_bytes(ctypes.byref(p))
    assert decode(sa, p, q=A, o=A, n=need) == INVALID


def test_the_binding_refuses_host_tensors(sa):
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i = torch.zeros((1, 2), dtype=torch.int32)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        sa.sa_cache_append(z(1, 1, 2, 64), z(1, 1, 2, 64), z(3, 2, 64, 64), z(3, 2, 64, 64), i, n)
    with pytest.raises(ValueError):
        sa.sa_route_pages(z(1, 1, 2, 64), torch.zeros(3, 2, 64), i, n, 0, 4)
    with pytest.raises(ValueError):
        sa.sa_attn_decode(z(1, 1, 2, 64), z(3, 2, 64, 64), z(3, 2, 64, 64), i, n)


def test_the_binding_refuses_unlike_caches(sa):
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)
    i = torch.zeros((1, 2), dtype=torch.int32)
    ok = z(3, 2, 64, 64)
    p = sa.make_cache_params(i, q=z(1, 1, 4, 64), k_cache=ok, v_cache=ok)
    assert (p.B, p.S, p.H, p.H_kv, p.D, p.n_pages, p.max_pages) == (1, 1, 4, 2, 64, 3, 2)
    for k, v in ((ok, z(3, 2, 64, 128)), (z(3, 2, 32, 64), z(3, 2, 32, 64)),
                 (ok, ok.to(torch.float8_e4m3fn)), (ok.float(), ok.float()),
                 (ok.transpose(2, 3), ok.transpose(2, 3))):
        with pytest.raises(ValueError):
            sa.make_cache_params(i, q=z(1, 1, 4, 64), k_cache=k, v_cache=v)
    with pytest.raises(ValueError):
        sa.make_cache_params(i, q=z(1, 1, 4, 64))
    with pytest.raises(ValueError):
        sa.make_cache_params(i, q=z(1, 4, 64), k_cache=ok, v_cache=ok)
    f8 = sa.make_cache_params(i, k_cache=ok.to(torch.float8_e4m3fn), v_cache=ok.to(torch.float8_e4m3fn))
    assert f8.cache_format == sa.SA_CACHE_FP8


# ------------------------------------------------------------------- oracle --

def test_oracle_rotation_keeps_lengths_and_pairs():
    rng = np.random.default_rng(0)
    x, ang = rng.standard_normal((5, 8)), rng.standard_normal((5, 4))
    for layout in ("interleaved", "half"):
        y, _ = turn_ref(x, False, 0, np.cos(ang), np.sin(ang), layout)
        assert np.allclose(np.linalg.norm(y, axis=1), np.linalg.norm(x, axis=1))
    y, _ = turn_ref(np.array([[1.0, 0, 0, 0]]), False, 0, np.array([[0.0, 1]]), np.array([[1.0, 0]]), "half")
    assert np.allclose(y, [[0, 0, 1, 0]])                       # (x0, x2) turned by a right angle
    n, _ = turn_ref(x, None, 0.0, None, None, "half")
    assert np.allclose(np.mean(n * n, axis=1), 1)


def test_oracle_places():
    got = list(places([62, 0, 127], [3, 0, 9], 5, 2))
    assert got == [(0, 0, 62), (0, 1, 63), (0, 2, 64), (2, 0, 127)]


def test_oracle_route_by_hand():
    # one row of five pages with scores 3, 1, 2, 1, 9; the newest is kept whatever it scores
    k_sum = np.array([3.0, 1, 2, 1, 9])[:, None, None]
    q, table = np.ones((1, 1, 1)), np.arange(5)[None]
    f = lambda prefix, budget, n=300: route_pages_ref(q, k_sum, table, [n], prefix, budget)[0]
    assert f(0, 2) == [0, 4] and f(0, 4) == [0, 1, 2, 4] and f(0, 0) == [4] and f(65, 0) == [0, 1, 4]
    assert f(0, 3, 129) == [0, 1, 2] and f(0, 3, 0) == [] and f(1000, 0) == [0, 1, 2, 3, 4]


def test_oracle_decode_is_softmax_attention():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 4, 2, 64, 8))
    q = rng.standard_normal((1, 4, 8))
    o, lse, _ = decode_ref(q, k, v, np.array([[2, 0, -1]]), [100], 0.3)
    kk = np.concatenate([k[2, 1], k[0, 1, :36]])
    vv = np.concatenate([v[2, 1], v[0, 1, :36]])
    x = 0.3 * kk @ q[0, 3]
    assert math.isclose(lse[0, 3], np.log(np.exp(x).sum()))
    assert np.allclose(o[0, 3], np.exp(x) / np.exp(x).sum() @ vv)
