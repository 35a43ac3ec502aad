"""Shared by the paged-cache tests: caches of a given storage and layout, and
the values they stand for."""

from __future__ import annotations

import numpy as np
import torch

PAGE = 64


def new_cache(n_pages, Hkv, D, fmt, layout="page_head", fill=None, gen=None, device="cuda"):
    """k_cache or v_cache [n_pages, Hkv, 64, D]: "page_head" contiguous,
    "page_token" with the token axis before the heads in memory, "gapped" a
    slice of a larger buffer. Returns (cache, its whole buffer)."""
    dt = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
    shape = {"page_head": (n_pages, Hkv, PAGE, D), "page_token": (n_pages, PAGE, Hkv, D),
             "gapped": (n_pages + 1, Hkv + 2, PAGE + 1, D + 16)}[layout]
    x = torch.zeros(shape) if fill is None else torch.randn(shape, generator=gen) * fill
    buf = x.to(dt).to(device)
    t = buf
    if layout == "page_token":
        t = buf.permute(0, 2, 1, 3)
    elif layout == "gapped":
        t = buf[:n_pages, 1:Hkv + 1, :PAGE, :D]
    return t, buf


def values(cache, scale=None):
    """What a cache stands for, fp64 on the host."""
    x = cache.detach().cpu().contiguous()
    x = x.view(torch.uint8).view(x.dtype).float().double().numpy()
    return x if scale is None else x * scale.cpu().double().numpy()[None, :, None, None]


def raw(t):
    """The bytes of a tensor, on the host."""
    return t.detach().cpu().contiguous().view(torch.uint8).numpy()


def page_table(lens, max_pages, n_pages, gen, fill=-1):
    """Distinct pages in no order for sequences of `lens` tokens."""
    perm = torch.randperm(n_pages, generator=gen).tolist()
    table = np.full((len(lens), max_pages), fill, dtype=np.int32)
    for b, n in enumerate(lens):
        for j in range(min(max_pages, (max(n, 0) + PAGE - 1) // PAGE)):
            table[b, j] = perm.pop()
    return table


def dev(a, dtype=torch.int32):
    return None if a is None else torch.as_tensor(np.asarray(a), dtype=dtype).cuda()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")
