"""fp64 reference of the paged key-value cache: appending with QK-norm and
rotation, the page router, and the attention of one new token.

Plain NumPy, written from the definitions and sharing no code with the CUDA
library. Tensors are NumPy arrays: keys and values of the caches as the values
they stand for (code * scale), page tables and lengths as integers.
"""

from __future__ import annotations

import math

import numpy as np

PAGE = 64


def turn_ref(x, gamma, eps, cos, sin, layout):
    """QK-norm (gamma is not False) and rotation (cos is not None) of x [..., D]
    in fp64; cos, sin [..., D/2] broadcast against x without its last axis.
    Also returns the magnitude of the terms each output was summed from."""
    y = np.asarray(x, dtype=np.float64)
    D = y.shape[-1]
    if gamma is not False:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps)
        if gamma is not None:
            y = y * gamma
    if cos is None:
        return y, np.abs(y)
    i = np.arange(D // 2)
    a, b = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + D // 2)
    out, mag = np.empty_like(y), np.empty_like(y)
    out[..., a] = y[..., a] * cos - y[..., b] * sin
    out[..., b] = y[..., a] * sin + y[..., b] * cos
    mag[..., a] = np.abs(y[..., a] * cos) + np.abs(y[..., b] * sin)
    mag[..., b] = np.abs(y[..., a] * sin) + np.abs(y[..., b] * cos)
    return out, mag


def places(seq_lens, new_lens, S, max_pages):
    """(sequence, token, position) of every new token that finds a place."""
    for b, n0 in enumerate(seq_lens):
        n0 = min(max(int(n0), 0), PAGE * max_pages)
        n = S if new_lens is None else min(max(int(new_lens[b]), 0), S)
        for s in range(min(n, PAGE * max_pages - n0)):
            yield b, s, n0 + s


def page_scores(q, k_sum, table, n, g):
    """Scores of one row's pages: max over the head group of q_h . k_sum; a
    page with a bad id, or no number for a score, gives -inf. q [G, D]."""
    nb = (n + PAGE - 1) // PAGE
    out = np.full(nb, -math.inf)
    for j in range(nb):
        if 0 <= table[j] < k_sum.shape[0]:
            s = q.astype(np.float64) @ k_sum[table[j], g].astype(np.float64)
            s = s[~np.isnan(s)]
            if s.size:
                out[j] = s.max()
    return out


def route_pages_ref(q, k_sum, table, seq_lens, prefix, budget):
    """Lists of kept pages per row b*H_kv + g. q [B, H, D]."""
    B, H, _ = q.shape
    Hkv, max_pages = k_sum.shape[1], table.shape[1]
    G, rows = H // Hkv, []
    for b in range(B):
        n = min(max(int(seq_lens[b]), 0), PAGE * max_pages)
        nb = (n + PAGE - 1) // PAGE
        for g in range(Hkv):
            forced = set(range((min(prefix, n) + PAGE - 1) // PAGE)) | ({nb - 1} if nb else set())
            s = page_scores(q[b, g * G:(g + 1) * G], k_sum, table[b], n, g)
            free = sorted((j for j in range(nb) if j not in forced), key=lambda j: (-s[j], j))
            rows.append(sorted(forced | set(free[:max(0, min(nb, budget) - len(forced))])))
    return rows


def decode_ref(q, k, v, table, seq_lens, scale, rows=None):
    """o [B, H, D], lse [B, H] and sum_u a_u |v_u| of one new token per
    sequence; k, v [n_pages, H_kv, 64, D]; rows: page lists per b*H_kv + g."""
    B, H, D = q.shape
    Hkv, G, max_pages = k.shape[1], H // k.shape[1], table.shape[1]
    o, lse, mag = np.zeros((B, H, D)), np.full((B, H), -math.inf), np.zeros((B, H, D))
    for b in range(B):
        n = min(max(int(seq_lens[b]), 0), PAGE * max_pages)
        for g in range(Hkv):
            js = range((n + PAGE - 1) // PAGE) if rows is None else rows[b * Hkv + g]
            js = [j for j in js if 0 <= table[b][j] < k.shape[0]]
            if not js:
                continue
            ks = np.concatenate([k[table[b][j], g, :min(PAGE, n - PAGE * j)] for j in js])
            vs = np.concatenate([v[table[b][j], g, :min(PAGE, n - PAGE * j)] for j in js])
            x = scale * (q[b, g * G:(g + 1) * G].astype(np.float64) @ ks.T)
            m = x.max(axis=1, keepdims=True)
            e = np.exp(x - m)
            z = e.sum(axis=1, keepdims=True)
            o[b, g * G:(g + 1) * G] = e / z @ vs
            mag[b, g * G:(g + 1) * G] = e / z @ np.abs(vs)
            lse[b, g * G:(g + 1) * G] = (m + np.log(z))[:, 0]
    return o, lse, mag
