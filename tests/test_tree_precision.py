"""sa_attn_tree where the weights' own precision shows, and over long contexts where each key
does.

A weight alone. As for one token (test_cache_decode_precision.py): one cached key has a logit
below the others', and its value is cancelled, column by column, by values of keys of weight 1,
so that the output is the error of that one weight, seen against the magnitudes that cancel.
Every new token stands alone: it sees the context and itself (a key and a value of zeros).
Every product q k here is exact, so a logit is off by its scaling only, 2^-23 |l|, and a weight
by that and by the exponential and its argument's rounding, 2^-21 for both: 2 dl. The weight
then goes into the product in terms:
  up to 16 rows a key-value head                2^-21 of it,
  more, bf16: 8 bits cut, 8 bits rounded        2^-16 of it, and 2^-22 that is added
              to what is left and the rounding of that sum,
  more, e4m3: 11 bits rounded twice             2^-21 of it, or 2^-30 of the largest weight
              (half a step of fp16's least, 2^-25, of 2^5 weights).
A sum of n products and what is there already, added in 24 bits and perhaps cut, is off by
2^-23 of the magnitudes for each; there are two or three such sums, and that of the weights:
  |o - exact| <= 2^-8 |exact| + (2 dl + term + 4 (n + 1) 2^-23) sum a |v| + 2^-30 max a sum |v|.

Long contexts. Keys of zeros give every token one weight, values are small whole numbers and
sums of them whole numbers below 2^24, so every sum is exact but for the second term of a
weight in bf16: 2^-23 of it, in 7,044 products of 16 keys, each of which may cost what is there
already its last place, 2^-15 as the sums of a run stay below 2^9: 0.22. The values of a column
add up to at most 40 over the context and 128 over the new tokens, so the output's rounding is
0.66 at most, and a key that is left out, taken twice or taken from another place is a difference
of 1 or more."""

import math

import numpy as np
import pytest
import torch

from cache_helpers import PAGE, dev, new_cache, page_table, status, values
from helpers import lib
from oracle.tree_oracle import tree_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return lib()


def stored(x, dt):
    return float(torch.tensor(x, dtype=torch.float32).to(dt).float())


@pytest.mark.parametrize("S,H", [(1, 1), (4, 4), (3, 8), (4, 8), (5, 8), (16, 7), (43, 3), (64, 7)])
@pytest.mark.parametrize("max_pages", [2, 400])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_a_weight_alone(sa, fmt, D, max_pages, S, H):
    """1 to 448 rows on a key-value head; tables small and large, which choose the kernel for
    17 to 32."""
    dt, top, n = (torch.bfloat16, 1.0, 5) if fmt == "bf16" else (torch.float8_e4m3fn, 256.0, 7)
    B, rows = 4, S * H
    rng = np.random.default_rng(D + rows)
    gen = torch.Generator().manual_seed(rows)
    lens = [n] * B
    table = page_table([n + S] * B, max_pages, 2 * B + 1, gen)
    kc, _ = new_cache(2 * B + 1, 1, D, fmt)
    vc, _ = new_cache(2 * B + 1, 1, D, fmt)
    q = torch.zeros((B, S, H, D), dtype=torch.bfloat16)
    q[..., 0] = torch.tensor(-rng.uniform(0.05, 4.0, (B, S, H))).to(torch.bfloat16)
    own = np.arange(D) * rows // D if rows > D else np.arange(D) % rows      # a row for each column
    k, v = torch.zeros((2 * B + 1, 1, PAGE, D)), torch.zeros((2 * B + 1, 1, PAGE, D))
    for b in range(B):
        page = table[b, 0]
        k[page, 0, 0, 0] = 1.0                       # the others' logits are 0
        for d in range(D):
            p = math.exp(float(q[b, own[d] // H, own[d] % H, 0]))
            v[page, 0, 0, d] = stored(top * rng.uniform(1.0, 1.7), dt)
            left = p * float(v[page, 0, 0, d])
            for i in range(1, n):
                v[page, 0, i, d] = stored(-left, dt)
                left += float(v[page, 0, i, d])
    kc.copy_(k.to(dt).cuda())
    vc.copy_(v.to(dt).cuda())
    st = status()
    alone = dev(np.full((B, S), -1))
    o, lse = sa.sa_attn_tree(q.cuda(), kc, vc, dev(table), dev(lens), scale=1.0, parents=alone, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    vals = values(vc)
    eo, el, mag, _ = tree_ref(q.double().numpy(), values(kc), vals, table, lens, None,
                              np.full((B, S), -1), 1.0)
    dl = 2.0 ** -23 * np.abs(q[..., :1].double().numpy()) + 2.0 ** -22
    term = 2.0 ** -21 if rows <= 16 or fmt == "fp8" else 2.0 ** -16 + 2.0 ** -22
    tol = 2.0 ** -8 * np.abs(eo) + (2 * dl + term + 4 * (n + 2) * 2.0 ** -23) * mag
    if fmt == "fp8":
        total = np.stack([np.abs(vals[table[b, 0], 0, :n]).sum(0) for b in range(B)])
        largest = np.exp(-el.transpose(0, 2, 1))                             # 1 / the sum of the weights
        tol = tol + 2.0 ** -30 * largest[..., None] * total[:, None, None]
    # the case says something: what is left is below the tolerance of 16-bit weights
    d = np.arange(D)
    left = np.abs(eo[:, own // H, own % H, d]) / mag[:, own // H, own % H, d]
    assert np.median(left) < 2.0 ** -16
    got = o.cpu().double().numpy()
    assert np.all(np.abs(got - eo) <= tol), float(np.max(np.abs(got - eo) / tol))
    assert np.all(np.abs(lse.cpu().double().numpy() - el) <= 2.0 ** -20 * (np.abs(el) + 1))


@pytest.mark.parametrize("lens,S,G", [([112640], 64, 7), ([112639, 64, 30001], 16, 7), ([112600, 5], 4, 4),
                                      ([70000, 112577], 5, 5)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_every_key_of_a_long_context_counts_once(sa, fmt, D, lens, S, G):
    rng = np.random.default_rng(S + D)
    gen = torch.Generator().manual_seed(S)
    B, Hkv = len(lens), 2
    after = [n + S for n in lens]
    max_pages = -(-max(after) // PAGE)
    n_pages = sum(-(-n // PAGE) for n in after) + 1
    table = page_table(after, max_pages, n_pages, gen)
    kc, _ = new_cache(n_pages, Hkv, D, fmt)
    vc, _ = new_cache(n_pages, Hkv, D, fmt)
    sums = np.zeros((B, Hkv, S, D))
    for b, n in enumerate(lens):
        v = rng.integers(-2, 3, (n + S, Hkv, D))
        over = v[:n].sum(0)                                      # brought into [-40, 40] by single tokens
        for g in range(Hkv):
            for d in range(D):
                want = int(rng.integers(-40, 41))
                at = rng.permutation(n)
                for t in at:
                    if over[g, d] == want:
                        break
                    new = int(np.clip(v[t, g, d] + np.clip(want - over[g, d], -2, 2), -2, 2))
                    over[g, d] += new - v[t, g, d]
                    v[t, g, d] = new
        sums[b] = (v[:n].sum(0)[:, None] + np.cumsum(v[n:].transpose(1, 0, 2), 1))
        x = torch.zeros((-(-(n + S) // PAGE) * PAGE, Hkv, D))
        x[:n + S] = torch.from_numpy(v).float()
        pages = dev(table[b, :x.shape[0] // PAGE], torch.int64)
        x = x.reshape(-1, PAGE, Hkv, D).permute(0, 2, 1, 3).to(vc.dtype).cuda()
        if fmt == "fp8":
            vc.view(torch.uint8)[pages] = x.view(torch.uint8)
        else:
            vc[pages] = x
    q = torch.randn((B, S, Hkv * G, D), generator=gen).to(torch.bfloat16).cuda()
    st = status()
    o, lse = sa.sa_attn_tree(q, kc, vc, dev(table), dev(lens), dev_status=st)      # a chain
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    n = np.array(lens)[:, None] + np.arange(1, S + 1)                              # [B, S]
    got = o.cpu().double().numpy().reshape(B, S, Hkv, G, D) * n[:, :, None, None, None]
    exp = sums.transpose(0, 2, 1, 3)[:, :, :, None]
    off = np.abs(got - exp)
    assert np.all(off <= (2.0 ** -8 + 2.0 ** -21) * np.abs(exp) + 0.25), float(off.max())
    el = np.log(n)[:, None]
    assert np.all(np.abs(lse.cpu().double().numpy() - el) <= 2.0 ** -21 * (el + 1))
