"""fp64 reference of the calls on drafted tokens and on a pool's pages: attention of a
tree of new tokens, the accepted path, forked, resized and compacted page tables.

Plain NumPy and lists, written from the definitions and sharing no code with the CUDA
library. Caches are NumPy arrays of the values they stand for.
"""

from __future__ import annotations

import math

import numpy as np

PAGE = 64


def ancestors_ref(parents, n):
    """seen[s, a]: whether new token a is s or one that s continues. parents of the first
    n tokens, or None (each continues the one before it); one that does not come before
    its token counts as -1."""
    seen = np.zeros((n, n), dtype=bool)
    for s in range(n):
        a = s
        while a >= 0:
            seen[s, a] = True
            up = a - 1 if parents is None else int(parents[a])
            a = up if -1 <= up < a else -1
    return seen


def new_tokens_ref(seq_lens, new_lens, S, max_pages):
    """[(tokens before, new tokens with a place)] of every sequence."""
    out = []
    for b, n in enumerate(seq_lens):
        n = min(max(int(n), 0), PAGE * max_pages)
        m = S if new_lens is None else min(max(int(new_lens[b]), 0), S)
        out.append((n, min(m, PAGE * max_pages - n)))
    return out


def tree_ref(q, k, v, table, seq_lens, new_lens, parents, scale, rows=None):
    """o [B, S, H, D], lse [B, H, S], sum_u a_u |v_u| and which [B, S] tokens are written;
    q [B, S, H, D]; parents [B][S] or None; rows: page lists per b*H_kv + g."""
    B, S, H, D = q.shape
    Hkv, max_pages = k.shape[1], table.shape[1]
    G = H // Hkv
    o, mag = np.zeros((B, S, H, D)), np.zeros((B, S, H, D))
    lse, written = np.full((B, H, S), -math.inf), np.zeros((B, S), dtype=bool)
    for b, (base, n) in enumerate(new_tokens_ref(seq_lens, new_lens, S, max_pages)):
        if n == 0:
            continue
        written[b, :n] = True
        seen = ancestors_ref(None if parents is None else parents[b], n)
        own = range(base // PAGE, (base + n + PAGE - 1) // PAGE)
        for g in range(Hkv):
            listed = range(base // PAGE) if rows is None else \
                [j for j in rows[b * Hkv + g] if 0 <= j < base // PAGE]
            js = [j for j in list(listed) + list(own) if 0 <= table[b][j] < k.shape[0]]
            for s in range(n):
                at = [(table[b][j], t % PAGE) for j in js
                      for t in range(j * PAGE, min((j + 1) * PAGE, base + n))
                      if t < base or seen[s, t - base]]
                if not at:
                    continue
                page, slot = (np.array(x) for x in zip(*at))
                ks, vs = k[page, g, slot], v[page, g, slot]
                x = scale * (q[b, s, g * G:(g + 1) * G].astype(np.float64) @ ks.T)
                m = x.max(axis=1, keepdims=True)
                e = np.exp(x - m)
                z = e.sum(axis=1, keepdims=True)
                o[b, s, g * G:(g + 1) * G] = e / z @ vs
                mag[b, s, g * G:(g + 1) * G] = e / z @ np.abs(vs)
                lse[b, g * G:(g + 1) * G, s] = (m + np.log(z))[:, 0]
    return o, lse, mag, written


def path_ref(path, m, base, max_pages, most=64):
    """The part of a path that counts."""
    out = []
    for a in list(path)[:m]:
        if not (a > (out[-1] if out else -1) and a < most and base + a < PAGE * max_pages):
            break
        out.append(int(a))
    return out


def accept_ref(k, v, k_sum, table, seq_lens, path, path_lens, k_scale=None):
    """Moves the paths' tokens in k, v [n_pages, H_kv, 64, D] (as stored; changed) and
    renews k_sum; returns the new lengths."""
    max_pages, ends = table.shape[1], []
    good = lambda p: 0 <= p < k.shape[0]
    for b, n in enumerate(seq_lens):
        base = min(max(int(n), 0), PAGE * max_pages)
        walk = path_ref(path[b], min(max(int(path_lens[b]), 0), path.shape[1]), base, max_pages)
        for i, a in enumerate(walk):
            f, t = table[b][(base + a) // PAGE], table[b][(base + i) // PAGE]
            if good(f) and good(t):
                for x in (k, v):
                    x[t, :, (base + i) % PAGE] = x[f, :, (base + a) % PAGE]
        end = base + len(walk)
        ends.append(end)
        for j in range(base // PAGE, (end + PAGE - 1) // PAGE):
            if k_sum is not None and good(table[b][j]):
                s = k[table[b][j], :, :min(PAGE, end - j * PAGE)].sum(axis=1)
                k_sum[table[b][j]] = s if k_scale is None else s * k_scale[:, None]
    return ends


def fork_ref(table, seq_lens, refs, src):
    """(table_out, lens_out, refs_out, moves, whether a page was missing)."""
    B, max_pages = table.shape
    good = lambda p: 0 <= p < len(refs)
    free = [p for p, r in enumerate(refs) if r <= 0]
    refs_out, out, ends, moves, taken, short = np.array(refs), [], [], [], set(), False
    for b in range(B):
        for p in table[b]:
            if good(p):
                refs_out[p] -= 1
    for s in src:
        if not 0 <= s < B:
            out.append([-1] * max_pages)
            ends.append(0)
            continue
        n = min(max(int(seq_lens[s]), 0), PAGE * max_pages)
        row = [int(p) if good(p) else -1 for p in table[s]]
        if s in taken:
            whole = n // PAGE
            last = row[whole] if n % PAGE else -1
            row[whole:] = [-1] * (max_pages - whole)
            if last >= 0:
                if free:
                    row[whole] = free.pop(0)
                    moves.append((last, row[whole]))
                else:
                    short, n = True, whole * PAGE
        taken.add(s)
        out.append(row)
        ends.append(n)
    for row in out:
        for p in row:
            if p >= 0:
                refs_out[p] += 1
    return np.array(out), ends, refs_out, moves, short


def resize_ref(table, refs, want_lens):
    """(table, refs, whether a page or place was missing)."""
    table, refs, short = np.array(table), np.array(refs), False
    free = [p for p, r in enumerate(refs) if r <= 0]
    for b, n in enumerate(want_lens):
        want = (max(int(n), 0) + PAGE - 1) // PAGE
        short |= want > table.shape[1]
        for j in range(table.shape[1]):
            has = 0 <= table[b, j] < len(refs)
            if j < want and not has:
                table[b, j] = free.pop(0) if free else -1
                short |= table[b, j] < 0
                if table[b, j] >= 0:
                    refs[table[b, j]] = 1
            elif j >= want:
                if has:
                    refs[table[b, j]] -= 1
                table[b, j] = -1
    return table, refs, short


def compact_ref(table, refs):
    """(table, refs, moves, pages in use)."""
    refs = np.array(refs)
    used = [p for p, r in enumerate(refs) if r > 0]
    n = len(used)
    holes = [p for p in range(n) if refs[p] <= 0]
    moves = list(zip([p for p in used if p >= n], holes))
    now = dict(moves)
    out = np.array([[now.get(int(p), int(p)) if 0 <= p < len(refs) else -1 for p in row]
                    for row in table]).reshape(np.shape(table))
    after = refs.copy()
    for a, b in moves:
        after[b], after[a] = refs[a], 0
    return out, after, moves, n
