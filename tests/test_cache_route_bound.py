"""The error bound by which sa_route_pages calls a page decided.

Over |q|_1 max |k| of a page and a head: the two bf16 terms of a key sum leave at most
2^-17 of it (measured below over every mantissa). A step of 16 products and the running sum,
17 terms none of which is larger than |q|_1 max |k|, cuts each to a unit in the last place
of the largest, 2^-23 of it: D / 16 steps for each of the two terms, the second of
which is 2^-8 of the first; and one more rounding joins them."""

import os
import re

import numpy as np
import pytest
import torch

from cache_helpers import dev, page_table, status
from helpers import lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "block_sparse_attention_sa_gb300", "csrc", "route_pages.cu")


def k_err():
    with open(SOURCE) as f:
        m = re.search(r"constexpr float kErr = (0x[0-9a-f.]+p-\d+|1\.f / \d+\.)f;", f.read())
    return float.fromhex(m.group(1)) if m.group(1)[:2] == "0x" else 1 / float(m.group(1)[6:])


def split_error():
    """Largest error of a value as two bf16 terms, over the value: all mantissas of [1, 2)."""
    x = (np.arange(1 << 23, dtype=np.uint32) | np.uint32(0x3F800000)).view(np.float32)
    t = torch.from_numpy(x)
    hi = t.to(torch.bfloat16).float()
    lo = (t - hi).to(torch.bfloat16).float()
    return float(((t.double() - hi.double() - lo.double()) / t.double()).abs().max())


def test_the_bound_follows_from_its_parts():
    terms = split_error()
    assert terms <= 2.0 ** -17
    steps = 128 // 16
    sums = steps * 17 * 2.0 ** -23 * (1 + 2.0 ** -8)
    assert k_err() >= terms + sums + 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("signs", ["mixed", "equal"])
@pytest.mark.parametrize("H,Hkv,D", [(8, 2, 128), (8, 2, 64), (56, 1, 128)])
def test_scores_lie_within_the_bound(H, Hkv, D, signs):
    """Sums and queries of one magnitude but for the last bits, where |q|_1 max |k| is least.
    The scores stand at the head of the workspace, [B * H_kv][max_pages] fp32."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sa = lib()
    rng = np.random.default_rng(D + H)
    n_pages = 200
    sign = lambda *s: rng.choice([-1.0, 1.0], s) if signs == "mixed" else np.ones(s)
    ksum = ((2.0 - rng.integers(1, 1 << 12, (n_pages, Hkv, D)) * 2.0 ** -23)
            * sign(n_pages, Hkv, D)).astype(np.float32)
    q = torch.tensor((2.0 - 2.0 ** -7) * sign(1, 1, H, D)).to(torch.bfloat16)
    table = page_table([64 * n_pages], n_pages, n_pages, torch.Generator().manual_seed(1))
    lens, st = dev([64 * n_pages]), status()
    args = (q.cuda(), torch.from_numpy(ksum).cuda(), dev(table), lens)
    p = sa.make_cache_params(args[2], q=args[0], k_sum=args[1], budget=9)
    ws = torch.zeros(sa.sa_route_pages_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    sa.sa_route_pages(*args, 0, 9, workspace=ws, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    got = ws[:4 * Hkv * n_pages].view(torch.float32).view(Hkv, n_pages).cpu().double().numpy()
    qd, G = q[0, 0].double().numpy(), H // Hkv
    for g in range(Hkv):
        exact = (qd[g * G:(g + 1) * G] @ ksum[table[0], g].astype(np.float64).T).max(axis=0)
        size = np.abs(qd[g * G:(g + 1) * G]).sum(axis=1).max() * np.abs(ksum[table[0], g]).max(axis=1)
        assert np.all(np.abs(got[g] - exact) <= k_err() * size)
