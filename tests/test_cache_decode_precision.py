"""sa_attn_decode where the weights' own precision shows.

One key has a logit below the others', and its value is cancelled, column by column, by
values of keys of weight 1, each of which takes up what the ones before it leave. What
remains is next to nothing, so the output is the error of that one weight, seen against
the magnitudes that cancel: the final rounding of the output hides none of it.

Every product q k here is exact (one element of each is not zero), so a logit l is off by
its scaling only, and a weight by that and the exponential: dl = 2^-23 |l| + 2^-22. A
weight is then held to 2^-21 of itself (three terms of 8 bits that leave 2^-22, and 2^-23
that is added to keep them positive; two terms of 11 bits leave 2^-22), and the n terms of
a sum are added in fp32, a unit in the last place each. So
  |o - exact| <= 2^-8 |exact| + (2 dl + 2^-21 + 2 n 2^-23) sum a |v|."""

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


def stored(x, dt):
    return float(torch.tensor(x, dtype=torch.float32).to(dt).float())


@pytest.mark.parametrize("heads", [(8, 1), (16, 1), (24, 1), (56, 1)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_a_weight_alone(sa, fmt, D, heads):
    H, Hkv = heads
    dt, top, n = (torch.bfloat16, 1.0, 5) if fmt == "bf16" else (torch.float8_e4m3fn, 256.0, 7)
    B = 6
    rng = np.random.default_rng(D + H)
    gen = torch.Generator().manual_seed(H)
    lens = [n] * B
    table = page_table(lens, 1, B + 1, gen)
    kc, _ = new_cache(B + 1, Hkv, D, fmt)
    vc, _ = new_cache(B + 1, Hkv, D, fmt)
    q = torch.zeros((B, 1, H, D), dtype=torch.bfloat16)
    q[..., 0] = torch.tensor(-rng.uniform(0.05, 4.0, (B, 1, H))).to(torch.bfloat16)
    k, v = torch.zeros((B + 1, Hkv, PAGE, D)), torch.zeros((B + 1, Hkv, PAGE, D))
    for b in range(B):
        page = table[b, 0]
        k[page, 0, 0, 0] = 1.0                       # the others' logits are 0
        for d in range(D):
            p = math.exp(float(q[b, 0, d % H, 0]))
            v[page, 0, 0, d] = stored(top * rng.uniform(1.0, 1.7), dt)
            left = p * float(v[page, 0, 0, d])
            for i in range(1, n):
                v[page, 0, i, d] = stored(-left, dt)
                left += float(v[page, 0, i, d])
    kc.copy_(k.to(dt).cuda())
    vc.copy_(v.to(dt).cuda())
    st = status()
    o, lse = sa.sa_attn_decode(q.cuda(), kc, vc, dev(table), dev(lens), scale=1.0, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    eo, el, mag = decode_ref(q[:, 0].double().numpy(), values(kc), values(vc), table, lens, 1.0)
    dl = 2.0 ** -23 * np.abs(q[:, 0, :, :1].double().numpy()) + 2.0 ** -22
    tol = 2.0 ** -8 * np.abs(eo) + (2 * dl + 2.0 ** -21 + 2 * n * 2.0 ** -23) * mag
    # the case says something: what is left is below the tolerance of 16-bit weights
    own = np.abs(eo[:, np.arange(D) % H, np.arange(D)]) / mag[:, np.arange(D) % H, np.arange(D)]
    assert np.median(own) < 2.0 ** -16
    got = o[:, 0].cpu().double().numpy()
    assert np.all(np.abs(got - eo) <= tol), float(np.max(np.abs(got - eo) / tol))


@pytest.mark.parametrize("H,Hkv", [(8, 1), (16, 1), (32, 1), (56, 1)])
def test_infinite_values_meet_no_term_of_zero(sa, H, Hkv):
    """A weight that few bits hold, 1 among them, has terms that would be zero."""
    gen = torch.Generator().manual_seed(3)
    n, D = 150, 64
    table = page_table([n], 3, 4, gen)
    kc, _ = new_cache(4, Hkv, D, "bf16")
    vc, _ = new_cache(4, Hkv, D, "bf16", fill=1.0, gen=gen)
    vc[int(table[0, 0]), 0, 7, 5] = float("inf")
    vc[int(table[0, 2]), 0, 21, 6] = float("-inf")
    q = torch.randn((1, 1, H, D), generator=gen).to(torch.bfloat16).cuda()
    o, lse = sa.sa_attn_decode(q, kc, vc, dev(table), dev([n]))     # keys of zeros: all weights 1
    torch.cuda.synchronize()
    assert torch.all(o[..., 5] == float("inf")) and torch.all(o[..., 6] == float("-inf"))
    rest = [d for d in range(D) if d not in (5, 6)]
    assert torch.isfinite(o[..., rest]).all() and torch.isfinite(lse).all()
