"""sa_qk_prologue with axes (or without the norm) under both pooling blocks: the outputs do
not depend on the block, are the fp64 definition within the bounds of test_rope_axes.py, and
the block means are those of the outputs, so that the routes agree."""

import pytest
import torch

from cache_helpers import status
from helpers import lib
from oracle.cache_oracle import turn_ref
from test_cache_append import check_stored
from test_rope_axes import angles, axis_list, n_axes, some_tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return lib()


@pytest.mark.parametrize("S", [1, 63, 64, 65, 72, 73, 127, 128, 129, 191, 192, 193, 200, 256, 300, 1000])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("axes,D,B,H", [((16, 24, 24), 128, 1, 9), ((5, 9, 3), 64, 2, 3)], ids=str)
def test_blocks_of_64_and_128(sa, axes, D, B, H, norm, S):
    gen = torch.Generator().manual_seed(S + D)
    q, k = (torch.randn((B, S, H, D), generator=gen).to(torch.bfloat16) for _ in range(2))
    g = [1 + 0.1 * torch.randn(D, generator=gen) for _ in range(2)] if norm else [None, None]
    cos, sin = some_tables(50, D, gen)
    pos = torch.randint(0, 50, (B, S, n_axes(axes, D)), generator=gen, dtype=torch.int32)
    c = lambda t: None if t is None else t.cuda()
    st = status()
    args = dict(gamma_q=c(g[0]), gamma_k=c(g[1]), cos=c(cos), sin=c(sin), qk_norm=norm,
                positions=c(pos), axes=axes, dev_status=st)
    q64, k64, _ = sa.sa_qk_prologue(c(q), c(k), q_block=64, **args)
    qo, ko, ws = sa.sa_qk_prologue(c(q), c(k), q_block=128, **args)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.equal(qo, q64) and torch.equal(ko, k64)
    co, si = angles(cos.double().numpy(), sin.double().numpy(), pos.numpy(), axis_list(axes, D))
    for x, gamma, got in ((q, g[0], qo), (k, g[1], ko)):
        y, mag = turn_ref(x.double().numpy(), gamma.double().numpy() if norm else False, 1e-6,
                          co[:, :, None], si[:, :, None], "interleaved")
        check_stored(got.cpu().double().numpy(), y, mag, "bf16", None)
    got = sa.sa_route_pooled(qo, ws, prefix_len=min(S, 3), tau=1.0, q_block=128)
    exp = sa.sa_route(qo, ko, min(S, 3), 1.0, q_block=128)
    assert torch.equal(got[0], exp[0])
    nnz = int(exp[0][-1])
    assert torch.equal(got[1][:nnz], exp[1][:nnz])
    # in place
    q2, k2 = c(q).clone(), c(k).clone()
    sa.sa_qk_prologue(q2, k2, q_block=128, q_out=q2, k_out=k2, **args)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)


def test_what_lies_behind_a_sequence_is_not_read(sa):
    """A view whose buffer goes on with no numbers: nothing of them comes into the outputs,
    the means or the route; the norm left out, tables by place."""
    gen = torch.Generator().manual_seed(5)
    B, S, H, D = 2, 199, 3, 64
    wide = torch.randn((2, B, S + 16, H, D), generator=gen).to(torch.bfloat16).cuda()
    wide[:, :, S:] = float("nan")
    q, k = wide[0, :, :S], wide[1, :, :S]
    cos, sin = (t.cuda() for t in some_tables(S, D, gen))
    for block in (64, 128):
        qo, ko, ws = sa.sa_qk_prologue(q, k, cos=cos, sin=sin, qk_norm=False, q_block=block)
        q1, k1, w1 = sa.sa_qk_prologue(q.contiguous(), k.contiguous(), cos=cos, sin=sin,
                                       qk_norm=False, q_block=block)
        assert torch.equal(qo, q1) and torch.equal(ko, k1)
        assert bool(torch.isfinite(qo).all()) and bool(torch.isfinite(ko).all())
        got = sa.sa_route_pooled(qo, ws, 0, 1.0, k=ko, q_block=block)
        exp = sa.sa_route_pooled(q1, w1, 0, 1.0, k=k1, q_block=block)
        nnz = int(exp[0][-1])
        assert torch.equal(got[0], exp[0]) and torch.equal(got[1][:nnz], exp[1][:nnz])
