"""e4m3 codes of appended keys and values next to the middle between two codes: each is the
code nearest to the fp32 quotient of value and scale (ties to even), not to the product with
a rounded reciprocal, which may lie on the other side."""

import numpy as np
import pytest
import torch

from cache_helpers import PAGE, dev, new_cache
from helpers import lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return lib()


def codes(x):
    """Nearest e4m3 codes of fp32 values, saturating, as bytes."""
    t = torch.from_numpy(np.ascontiguousarray(np.clip(x, -448.0, 448.0)))
    return t.to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def hard(n, rng):
    """(value in bf16, scale in fp32) whose quotient and whose product with the reciprocal
    have different codes; middles of normal and of subnormal codes among them."""
    vals, scales = [], []
    while len(vals) < n:
        x = torch.tensor(rng.uniform(0.1, 4.0, 4096) * rng.choice([-1, 1], 4096)).bfloat16().float().numpy()
        code = rng.integers(0, 126, 4096)                       # below the largest
        mid = [torch.tensor([c, c + 1], dtype=torch.uint8).view(torch.float8_e4m3fn).double().mean().item()
               for c in code]
        s = (np.abs(x) / np.array(mid)).astype(np.float32)
        s = np.nextafter(s, np.where(rng.random(4096) < 0.5, 0, 9).astype(np.float32))
        differ = codes(x / s) != codes(x * (np.float32(1) / s))
        vals += x[differ].tolist()
        scales += s[differ].tolist()
    return np.array(vals[:n], dtype=np.float32), np.array(scales[:n], dtype=np.float32)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S", [1, 70])
def test_codes_next_to_the_middle(sa, S, D):
    Hkv = 48
    rng = np.random.default_rng(S + D)
    vals, scales = hard(Hkv, rng)
    assert np.any(np.abs(vals / scales) < 2.0 ** -6) and np.any(np.abs(vals / scales) > 2.0 ** -5)
    x = torch.randn((1, S, Hkv, D), generator=torch.Generator().manual_seed(S)).to(torch.bfloat16)
    for i in range(0, D, 7):                   # lanes with one such value, and with none
        x[0, :, :, i] = torch.from_numpy(vals)[None].to(torch.bfloat16)
    kc, _ = new_cache(3, Hkv, D, "fp8")
    vc, _ = new_cache(3, Hkv, D, "fp8")
    s = torch.from_numpy(scales).cuda()
    xd = x.cuda()
    for rope in ("interleaved", "half"):       # keys without norm and rotation, either layout of lanes
        kc.view(torch.uint8).fill_(0)
        sa.sa_cache_append(xd, xd, kc, vc, dev([[1, 2]]), dev([0]), k_scale=s, v_scale=s, rope=rope)
        torch.cuda.synchronize()
        want = codes(x[0].float().numpy() / scales[:, None])
        for c in (kc, vc):
            got = torch.cat([c[1], c[2]], dim=1)[:, :S].contiguous().view(torch.uint8).cpu().numpy()
            assert np.array_equal(got.transpose(1, 0, 2), want)


def test_powers_of_two_and_no_scale(sa):
    """Quotients that are exact, ties among them."""
    x = torch.arange(-64, 64).repeat(8, 1).to(torch.bfloat16) * torch.tensor([[2.0 ** i] for i in range(8)]).bfloat16()
    x = x.reshape(1, 8, 2, 64).cuda()
    for scale in (None, 0.25, 2.0 ** -9):
        kc, _ = new_cache(2, 2, 64, "fp8")
        vc, _ = new_cache(2, 2, 64, "fp8")
        s = None if scale is None else torch.full((2,), scale, device="cuda")
        sa.sa_cache_append(x, x, kc, vc, dev([[1]]), dev([0]), k_scale=s, v_scale=s)
        torch.cuda.synchronize()
        want = codes(x[0].float().cpu().numpy() / np.float32(scale or 1.0))
        for c in (kc, vc):
            got = c[1][:, :8].contiguous().view(torch.uint8).cpu().numpy().transpose(1, 0, 2)
            assert np.array_equal(got, want)
