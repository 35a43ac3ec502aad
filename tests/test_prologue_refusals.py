"""sa_qk_prologue, with and without axes, refuses what its kernels would read or write beyond."""

import pytest
import torch

from helpers import lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return lib()


@pytest.mark.parametrize("by_axes", [False, True])
def test_shapes_types_and_devices(sa, by_axes):
    S, H, D = 70, 3, 64
    x = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    f = lambda *s: torch.zeros(s, device="cuda")
    q, k = x(1, S, H, D), x(1, S, H, D)
    kw = dict(gamma_q=f(D), gamma_k=f(D), cos=f(S, D // 2), sin=f(S, D // 2),
              dev_status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if by_axes:
        kw["axes"] = (16, 16)
    sa.sa_qk_prologue(q, k, **kw)
    for a, b in ((q, k[:, :S - 1]), (q, k[:, :, :2]), (q, x(1, S, H, 128)[..., :32]), (q.float(), k.float()),
                 (q, k.half()), (q[0], k[0]), (torch.cat([q, q]), k)):
        with pytest.raises(ValueError):
            sa.sa_qk_prologue(a, b, **kw)
    # the strides of q, but not all of its tokens or heads
    wide = x(1, S, H, D)
    short = [dict(cos=f(S - 1, D // 2), sin=f(S - 1, D // 2))] if not by_axes else \
        [dict(cos=f(S, D // 4)), dict(positions=torch.zeros((1, S - 1, 2), dtype=torch.int32, device="cuda"))]
    for bad in [dict(q_out=wide[:, :S - 1]), dict(k_out=wide[:, :, :2]), dict(q_out=wide.half()),
                dict(gamma_q=f(D - 4)), dict(gamma_k=f(D // 2)), dict(dev_status=f(1)),
                dict(dev_status=torch.zeros(1, dtype=torch.int32)), dict(q_out=torch.zeros_like(q, device="cpu")),
                dict(workspace=torch.zeros(1 << 20, dtype=torch.uint8))] + short:
        with pytest.raises(ValueError):
            sa.sa_qk_prologue(q, k, **{**kw, **bad})
    # larger ones serve
    got = sa.sa_qk_prologue(q, k, **{**kw, "cos": f(S + 5, D // 2), "sin": f(S + 5, D // 2), "gamma_q": f(2 * D)})
    assert got[0].shape == q.shape
    torch.cuda.synchronize()
