"""Cases and plain forms of the operators of speculative decoding and of page
upkeep over the paged key-value cache, and of rotary positions with axes.

    tree     sa_attn_tree: attention of the drafted tokens of a tree over the
             cached pages, every page or the pages of a route
    accept   sa_cache_accept: the tokens of the verified path move together in
             the cache, the sums of their pages are made anew
    fork     sa_pages_fork, sa_pages_resize, sa_cache_copy: sequences are forked,
             reordered and dropped, and get pages for their next tokens
    compact  sa_pages_compact, sa_cache_copy: pages in use move to the pool's front
    axes     sa_qk_prologue or sa_cache_append with positions on several axes
             (time, height, width)

``run`` computes them in their plain form (elementary torch operations), or
through the framework where ``own`` is true. Sizes are those of the framework's
workloads (56 heads of 128, 38,247 / 112,640 / 8,192 tokens, prefix 951) and
common serving shapes (32 query heads on 8 key-value heads).
"""

import math

import torch

own = False

DEVICE = "cuda"
PAGE = 64
E4M3_MAX = 448.0


def listed():
    return [
        # one user, a small draft behind a short context: the latency of a call
        dict(name="tree one", op="tree", B=1, S=8, H=32, Hkv=8, D=128, fmt="bf16", past=777,
             ragged=False, budget=0, chain=False),
        # a serving batch of unequal lengths, unequal trees
        dict(name="tree batch", op="tree", B=32, S=16, H=56, Hkv=8, D=128, fmt="bf16", past=8192,
             ragged=True, budget=0, chain=False),
        # full trees behind a few very long contexts in 8 bits
        dict(name="tree long", op="tree", B=3, S=64, H=56, Hkv=8, D=128, fmt="fp8", past=112640,
             ragged=False, budget=0, chain=False),
        # the routed form, an odd number of drafted tokens in a row: 96 of 598 pages
        dict(name="tree routed", op="tree", B=24, S=5, H=16, Hkv=16, D=64, fmt="bf16", past=38247,
             ragged=True, budget=96, chain=True),
        # one user's path of a small tree
        dict(name="accept one", op="accept", B=1, S=8, Hkv=8, D=128, fmt="bf16", past=777,
             ragged=False),
        # the paths of a batch, 8-bit cache
        dict(name="accept batch", op="accept", B=128, S=64, Hkv=8, D=128, fmt="fp8", past=8192,
             ragged=True),
        # four beams of one user
        dict(name="fork beams", op="fork", B=4, N=4, Hkv=8, D=128, fmt="bf16", past=777,
             ragged=False),
        # a batch of many: some sequences end, others are continued several times
        dict(name="fork batch", op="fork", B=256, N=256, Hkv=8, D=128, fmt="bf16", past=2048,
             ragged=True),
        # a small pool
        dict(name="compact small", op="compact", B=4, Hkv=8, D=64, fmt="fp8", past=2000,
             ragged=True, fill=1.0),
        # a pool of a few GB, a third of it holes
        dict(name="compact pool", op="compact", B=48, Hkv=8, D=128, fmt="bf16", past=8192,
             ragged=True, fill=1.0),
        # one decoding step of a batch whose prompts hold images, 8-bit cache
        dict(name="axes append", op="axes", into="cache", B=128, S=1, H=32, Hkv=8, D=128,
             fmt="fp8", rope="half", norm=False, past=4095, ragged=True, t=16, h=24, w=24),
        # the packed release sequence: a prefix, then frames of a video
        dict(name="axes packed", op="axes", into="packed", B=1, S=38247, H=56, Hkv=56, D=128,
             rope="interleaved", norm=True, ragged=False, t=16, h=24, w=24, prefix=951),
    ]


HEADS = [(32, 8), (56, 8), (16, 16), (56, 1), (40, 10), (24, 4), (8, 2), (5, 5)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "accept", "fork", "compact", "axes"])
    H, Hkv = rng.choice(HEADS)
    D = rng.choice([64, 128, 128])
    case = dict(op=op, Hkv=Hkv, D=D, fmt=rng.choice(["bf16", "fp8"]), ragged=rng.random() < 0.6)
    if op in ("tree", "accept"):
        case["S"] = _log(rng, 1, 64)
    if op == "tree":
        case.update(H=H, past=_log(rng, 1, 112640), chain=rng.random() < 0.3,
                    budget=_log(rng, 1, 512) if rng.random() < 0.3 else 0)
        # 1 GB of keys and values in bf16, and no more work than the longest case
        most = min((1 << 30) // (case["past"] * Hkv * D * 4),
                   int(6e11 / (4.0 * case["S"] * H * D * case["past"])))
        case["B"] = _log(rng, 1, max(1, min(128, most)))
    elif op == "axes":
        case.update(H=H, rope=rng.choice(["interleaved", "half"]), norm=rng.random() < 0.5)
        t = rng.randint(1, D // 4)
        h = rng.randint(1, D // 2 - t - 1)
        # the pairs behind the last axis stay as they are
        case.update(t=t, h=h, w=rng.choice([D // 2 - t - h, rng.randint(1, D // 2 - t - h)]))
        if rng.random() < 0.5:
            case.update(into="packed", rope="interleaved", Hkv=H, S=_log(rng, 1, 38247),
                        ragged=False)
            case["B"] = _log(rng, 1, max(1, min(8, 38247 // case["S"])))
            case["prefix"] = rng.randint(0, min(951, case["S"]))
            del case["fmt"]
        else:
            case.update(into="cache", S=1 if rng.random() < 0.4 else _log(rng, 2, 8192))
            case["B"] = _log(rng, 1, max(1, min(256, 32768 // case["S"])))
            case["past"] = _log(rng, 1, 8192) - 1
    else:
        case.update(past=_log(rng, 1, 8192))
        most = (2 << 30) // (case["past"] * Hkv * D * 4)
        case["B"] = _log(rng, 1, max(1, min(256 if op != "compact" else 64, most)))
        if op == "fork":
            case["N"] = _log(rng, 1, 256)
        if op == "compact":
            case["fill"] = round(rng.uniform(0.3, 1.0), 2)
    return case


# ------------------------------------------------------------------ inputs --

def _lengths(case, gen):
    B, past = case["B"], case["past"]
    lens = torch.full((B,), past, dtype=torch.int32)
    if case["ragged"]:
        lens = (past * (0.25 + 0.75 * torch.rand((B,), generator=gen))).ceil().to(torch.int32)
        lens[int(torch.randint(0, B, (1,), generator=gen))] = past
    return lens


def _new_lens(case, gen):
    """How many new tokens each sequence of a padded batch brings."""
    if not case["ragged"] or case["S"] == 1:
        return None
    new = torch.randint(1, case["S"] + 1, (case["B"],), generator=gen, dtype=torch.int32)
    new[int(torch.randint(0, case["B"], (1,), generator=gen))] = case["S"]
    return new


def _pool(s, case, n_pages, gen, dev):
    """Unit-variance keys and values; in 8 bits codes with the heads' scales."""
    fp8 = case["fmt"] == "fp8"
    shape = (n_pages, case["Hkv"], PAGE, case["D"])
    s["ks"] = s["vs"] = None
    for name, sc in (("kc", "ks"), ("vc", "vs")):
        x = torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(generator=gen)
        if fp8:
            s[sc] = 0.02 + 0.02 * torch.rand((case["Hkv"],), generator=gen, device=dev)
            x = (x / s[sc].to(torch.bfloat16)[None, :, None, None]).clamp_(-E4M3_MAX, E4M3_MAX)
            x = x.to(torch.float8_e4m3fn)
        s[name] = x


def _sums(s, case, n_pages, gen, dev):
    shape = (n_pages, case["Hkv"], case["D"])
    s["ksum"] = torch.empty(shape, device=dev).normal_(0.0, 8.0, generator=gen)


def _spread_pages(lens, max_pages, n_pages, gen):
    """A table of pages in no order; -1 behind a sequence's last page."""
    need = (lens + PAGE - 1) // PAGE
    perm = torch.randperm(n_pages, generator=gen, dtype=torch.int64).to(torch.int32)
    table = torch.full((len(lens), max_pages), -1, dtype=torch.int32)
    used = torch.arange(max_pages)[None, :] < need[:, None]
    table[used] = perm[: int(need.sum())]
    return table


def prepare(case, seed):
    dev = torch.device(DEVICE)
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": dict(case)}
    {"tree": _prepare_tree, "accept": _prepare_accept, "fork": _prepare_fork,
     "compact": _prepare_compact, "axes": _prepare_axes}[case["op"]](s, case, host, gen, dev)
    return s


def _bf16(dev, gen, *shape, scale=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(0.0, scale, generator=gen)


def _behind(s, case, host, dev):
    """Sequences with S new tokens behind their `past` cached ones."""
    lens, new = _lengths(case, host), _new_lens(case, host)
    total = lens + (case["S"] if new is None else new)
    max_pages = (case["past"] + case["S"] + PAGE - 1) // PAGE
    n_pages = case["B"] * max_pages + 3
    table = _spread_pages(total, max_pages, n_pages, host)
    s.update(lens=lens.to(dev), new_lens=None if new is None else new.to(dev),
             table=table.to(dev))
    return n_pages, max_pages


def _prepare_tree(s, case, host, gen, dev):
    B, S, H, Hkv, D = case["B"], case["S"], case["H"], case["Hkv"], case["D"]
    n_pages, max_pages = _behind(s, case, host, dev)
    _pool(s, case, n_pages, gen, dev)
    s["q"] = _bf16(dev, gen, B, S, H, D, scale=2.0)
    s["parents"] = None
    if not case["chain"]:                      # each token continues some earlier one
        up = (torch.rand((B, S), generator=host) * torch.arange(S)[None, :]).floor()
        up[:, 0] = -1                          # the token that was sampled last
        s["parents"] = up.to(torch.int32).to(dev)
    s["row_ptr"] = s["col_idx"] = None
    if case["budget"]:
        _some_route(s, case, max_pages, gen, dev)
    s["o"] = torch.zeros((B, S, H, D), dtype=torch.bfloat16, device=dev)
    s["lse"] = torch.zeros((B, H, S), device=dev)


def _some_route(s, case, max_pages, gen, dev):
    """`budget` random pages of the context for each key-value head, ascending."""
    B, Hkv = case["B"], case["Hkv"]
    full = (s["lens"] // PAGE).long()[:, None, None]
    j = torch.arange(max_pages, device=dev)[None, None, :]
    score = torch.rand((B, Hkv, max_pages), generator=gen, device=dev).masked_fill(j >= full, -1.0)
    rank = score.argsort(-1, descending=True).argsort(-1)
    keep = ((rank < case["budget"]) & (j < full)).reshape(B * Hkv, max_pages)
    s["row_ptr"] = torch.zeros(B * Hkv + 1, dtype=torch.int32, device=dev)
    s["row_ptr"][1:] = keep.sum(-1).cumsum(0)
    s["col_idx"] = torch.full((max(1, B * Hkv * min(case["budget"], max_pages)),), -1,
                              dtype=torch.int32, device=dev)
    cols = keep.nonzero()[:, 1]
    s["col_idx"][: len(cols)] = cols.to(torch.int32)


def _prepare_accept(s, case, host, gen, dev):
    B, S = case["B"], case["S"]
    n_pages, _ = _behind(s, case, host, dev)
    _pool(s, case, n_pages, gen, dev)
    _sums(s, case, n_pages, gen, dev)
    # the first token and, of the others that a sequence has, some, in ascending order
    new = torch.full((B,), S, dtype=torch.int32) if s["new_lens"] is None else s["new_lens"].cpu()
    pick = torch.rand((B, S), generator=host) < 0.3
    pick[:, 0] = True
    pick &= torch.arange(S)[None, :] < new[:, None]
    order = torch.where(pick, torch.arange(S)[None, :], S).sort(-1).values
    s["path_lens"] = pick.sum(-1).to(torch.int32).to(dev)
    s["path"] = torch.where(order == S, -1, order).to(torch.int32).to(dev)
    s["lens_out"] = torch.zeros_like(s["lens"])


def _prepare_fork(s, case, host, gen, dev):
    B, N = case["B"], case["N"]
    lens = _lengths(case, host)
    max_pages = (case["past"] + PAGE) // PAGE + 1
    # groups of four sequences share the first half of the shortest one's full pages
    own_pages = _spread_pages(lens, max_pages, B * max_pages + N + 5, host)
    for b in range(0, B, 4):
        half = int(lens[b:b + 4].min()) // PAGE // 2
        own_pages[b:b + 4, :half] = own_pages[b, :half].clone()
    n_pages = B * max_pages + N + 5
    refs = torch.zeros(n_pages, dtype=torch.int32)
    held = own_pages[own_pages >= 0].long()
    refs.index_put_((held,), torch.ones_like(held, dtype=torch.int32), accumulate=True)
    _pool(s, case, n_pages, gen, dev)
    _sums(s, case, n_pages, gen, dev)
    # a few of the sequences have the better continuations; one place in sixteen is empty
    src = (B * torch.rand((N,), generator=host) ** 2).floor().clamp(max=B - 1).to(torch.int32)
    src[torch.rand((N,), generator=host) < 1 / 16] = -1
    s.update(table=own_pages.to(dev), lens=lens.to(dev), refs=refs.to(dev), src=src.to(dev),
             table_out=torch.full((N, max_pages), -1, dtype=torch.int32, device=dev),
             lens_out=torch.zeros(N, dtype=torch.int32, device=dev),
             refs_out=torch.zeros_like(refs).to(dev),
             moves=torch.full((N, 2), -1, dtype=torch.int32, device=dev),
             n_moves=torch.zeros(1, dtype=torch.int32, device=dev))


def _prepare_compact(s, case, host, gen, dev):
    lens = _lengths(case, host)
    max_pages = (case["past"] + PAGE - 1) // PAGE
    n_pages = int(math.ceil(case["B"] * max_pages / case["fill"]))
    table = _spread_pages(lens, max_pages, n_pages, host)
    refs = torch.zeros(n_pages, dtype=torch.int32)
    refs[table[table >= 0].long()] = 1
    _pool(s, case, n_pages, gen, dev)
    _sums(s, case, n_pages, gen, dev)
    s.update(table=table.to(dev), refs=refs.to(dev),
             table_out=torch.full_like(table, -1).to(dev), refs_out=torch.zeros_like(refs).to(dev),
             moves=torch.full((n_pages // 2 + 1, 2), -1, dtype=torch.int32, device=dev),
             n_moves=torch.zeros(1, dtype=torch.int32, device=dev),
             n_used=torch.zeros(1, dtype=torch.int32, device=dev))


def _grid_positions(S, prefix, start):
    """Positions (time, height, width) of `prefix` tokens of text and then frames
    of 24 x 42 patches; int32 [S, 3]."""
    i = torch.arange(S)
    text = i[:, None].expand(S, 3)
    j = (i - prefix).clamp(min=0)
    video = torch.stack((j // 1008, j // 42 % 24, j % 42), -1) + prefix
    return (start + torch.where((i < prefix)[:, None], text, video)).to(torch.int32)


def _prepare_axes(s, case, host, gen, dev):
    B, S, H, Hkv, D = case["B"], case["S"], case["H"], case["Hkv"], case["D"]
    s["q"], s["k"] = _bf16(dev, gen, B, S, H, D), _bf16(dev, gen, B, S, Hkv, D)
    s["gq"] = s["gk"] = None
    if case["norm"]:
        s["gq"] = 1 + 0.1 * _bf16(dev, gen, D).float()
        s["gk"] = 1 + 0.1 * _bf16(dev, gen, D).float()
    s["axes"] = (case["t"], case["h"], case["w"])
    s["q_out"] = torch.zeros_like(s["q"])
    if case["into"] == "packed":
        one = _grid_positions(S, case["prefix"], 0)
        s["positions"] = one[None].expand(B, S, 3).contiguous().to(dev)
        rows = int(one.max()) + 1
        s["k_out"] = torch.zeros_like(s["k"])
    else:
        n_pages, max_pages = _behind(s, case, host, dev)
        _pool(s, case, n_pages, gen, dev)
        _sums(s, case, n_pages, gen, dev)
        s["v"] = _bf16(dev, gen, B, S, Hkv, D)
        # images in the prompt use fewer positions than they have tokens
        start = (s["lens"].cpu() * (0.3 + 0.7 * torch.rand((B,), generator=host))).to(torch.int32)
        one = _grid_positions(S, min(S, 64), 0)
        s["positions"] = (one[None] + start[:, None, None]).contiguous().to(dev)
        rows = int(s["positions"].max()) + 1
        s["lens_out"] = torch.zeros_like(s["lens"])
    # frequencies of the pairs, each axis from its own first pair on
    size = torch.tensor(s["axes"] + (D // 2 - sum(s["axes"]),))
    axis_of = torch.repeat_interleave(torch.arange(4), size)
    within = torch.cat([torch.arange(int(n)) for n in size])
    freq = 1e4 ** (-within.double() / size[axis_of].clamp(min=1))
    angle = torch.arange(rows, dtype=torch.float64)[:, None] * freq
    s["cos"], s["sin"] = angle.cos().float().to(dev), angle.sin().float().to(dev)
    s["axis_of"] = axis_of.to(dev)


# -------------------------------------------------------------- plain forms --

def _bytes_of(cache):
    """Moved as bytes: torch indexes those everywhere."""
    return cache if cache.dtype == torch.bfloat16 else cache.view(torch.uint8)


def _ancestors(s, B, S, dev):
    """[B, S, S]: whether token a is token s or one that s continues."""
    if s["parents"] is None:
        return torch.ones((S, S), dtype=torch.bool, device=dev).tril_().expand(B, S, S)
    up = torch.zeros((B, S, S), device=dev)
    one = torch.eye(S, device=dev).expand(B, S, S)
    up.scatter_(2, s["parents"].clamp(min=0).long()[..., None], (s["parents"] >= 0).float()[..., None])
    reach = one + up
    for _ in range(max(1, (S - 1).bit_length())):
        reach = torch.matmul(reach, reach).clamp_(max=1.0)
    return reach > 0


def _tree_plain(s):
    c = s["case"]
    B, S, H, Hkv, D = c["B"], c["S"], c["H"], c["Hkv"], c["D"]
    G, dev = H // Hkv, s["q"].device
    n = s["table"].shape[1]
    page = s["table"].clamp(min=0).long()
    base = s["lens"].long()
    new = torch.full_like(base, S) if s["new_lens"] is None else s["new_lens"].long()
    keys = n * PAGE

    def values(cache, scale):
        x = _bytes_of(cache)[page].view(cache.dtype).permute(0, 2, 1, 3, 4).reshape(B, Hkv, keys, D)
        return x.float() if scale is None else x.float().mul_(scale[None, :, None, None])

    tok = torch.arange(keys, device=dev)
    at = tok[None, :] - base[:, None]                                     # [B, keys]
    mine = _ancestors(s, B, S, dev).gather(2, at.clamp(0, S - 1)[:, None, :].expand(B, S, keys))
    seen = (at < 0)[:, None, :] | (mine & ((at >= 0) & (at < new[:, None]))[:, None, :])
    seen = seen[:, None]                                                  # [B, 1, S, keys]
    if s["row_ptr"] is not None:
        row = torch.repeat_interleave(torch.arange(B * Hkv, device=dev),
                                      (s["row_ptr"][1:] - s["row_ptr"][:-1]).long())
        there = torch.zeros((B * Hkv, n), dtype=torch.bool, device=dev)
        there[row, s["col_idx"][: row.numel()].long()] = True
        there = there.view(B, Hkv, n) | (torch.arange(n, device=dev) >= base[:, None] // PAGE)[:, None]
        seen = seen & there.repeat_interleave(PAGE, -1)[:, :, None]
    qg = s["q"].view(B, S, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, S * G, D).float()
    logit = torch.matmul(qg, values(s["kc"], s["ks"]).transpose(-1, -2)).mul_(D ** -0.5)
    logit = logit.view(B, Hkv, S, G, keys).masked_fill_(~seen[:, :, :, None], -math.inf)
    top = logit.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = logit.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, S * G, keys), values(s["vc"], s["vs"])).view(B, Hkv, S, G, D)
    o = (o / total.clamp(min=1e-30)).permute(0, 2, 1, 3, 4).reshape(B, S, H, D)
    lse = (top + total.log())[..., 0].permute(0, 1, 3, 2).reshape(B, H, S)
    live = torch.arange(S, device=dev)[None, :] < new[:, None]
    s["o"].copy_(torch.where(live[:, :, None, None], o.to(torch.bfloat16), s["o"]))
    s["lse"].copy_(torch.where(live[:, None, :], lse, s["lse"]))


def _accept_plain(s):
    c = s["case"]
    B, S, Hkv, D = c["B"], c["S"], c["Hkv"], c["D"]
    dev = s["lens"].device
    base, n_acc = s["lens"].long(), s["path_lens"].long()
    i = torch.arange(S, device=dev)[None, :]
    b, i = (i < n_acc[:, None]).nonzero(as_tuple=True)
    frm, to = base[b] + s["path"][b, i].long(), base[b] + i
    for cache in (s["kc"], s["vc"]):
        x = _bytes_of(cache).permute(0, 2, 1, 3)                          # [page, slot, Hkv, D]
        moved = x[s["table"][b, frm // PAGE].long(), frm % PAGE]
        x[s["table"][b, to // PAGE].long(), to % PAGE] = moved
    # the pages from that of the old end to that of the new one
    end = base + n_acc
    j = torch.arange(s["table"].shape[1], device=dev)[None, :]
    b, j = ((j >= (base // PAGE)[:, None]) & (j * PAGE < end[:, None])).nonzero(as_tuple=True)
    page = s["table"][b, j].long()
    x = _bytes_of(s["kc"])[page].view(s["kc"].dtype).float()              # [pages, Hkv, 64, D]
    if s["ks"] is not None:
        x = x * s["ks"][None, :, None, None]
    live = (j[:, None] * PAGE + torch.arange(PAGE, device=dev)) < end[b][:, None]
    s["ksum"][page] = (x * live[:, None, :, None]).sum(2)
    s["lens_out"].copy_(end)


def _copy_plain(s):
    m = s["moves"][: int(s["n_moves"])].long()
    for cache in (_bytes_of(s["kc"]), _bytes_of(s["vc"]), s["ksum"]):
        cache[m[:, 1]] = cache[m[:, 0]]


def _count(refs, table, by):
    held = table[table >= 0].long()
    refs.index_put_((held,), torch.full_like(held, by, dtype=torch.int32), accumulate=True)


def _fork_plain(s):
    dev = s["src"].device
    src, refs, table = s["src"].long(), s["refs"], s["table"]
    N = len(src)
    there = src >= 0
    old = src.clamp(min=0)
    lens = torch.where(there, s["lens"][old], 0).long()
    out = torch.where(there[:, None], table[old], -1)
    # the first row that continues a sequence keeps its page in progress
    i = torch.arange(N, device=dev)
    first = torch.full((s["table"].shape[0],), N, device=dev).scatter_reduce_(
        0, old[there], i[there], "amin")
    again = there & (first[old] != i)
    behind = torch.arange(table.shape[1], device=dev)[None, :] >= (lens // PAGE)[:, None]
    out = out.masked_fill(again[:, None] & behind, -1)
    need = (again & (lens % PAGE > 0)).nonzero()[:, 0]
    fresh = (refs == 0).nonzero()[:, 0][: len(need)]
    place = lens[need] // PAGE
    s["moves"][: len(need), 0] = table[old[need], place]
    s["moves"][: len(need), 1] = fresh.to(torch.int32)
    s["n_moves"].fill_(len(need))
    out[need, place] = fresh.to(torch.int32)
    s["refs_out"].copy_(refs)
    _count(s["refs_out"], table, -1)
    _count(s["refs_out"], out, 1)
    s["lens_out"].copy_(lens)
    # room for one more token: pages behind that are given back, missing ones taken
    mine = torch.arange(table.shape[1], device=dev)[None, :] < ((lens + PAGE) // PAGE)[:, None]
    free = (s["refs_out"] == 0).nonzero()[:, 0]
    _count(s["refs_out"], out.masked_fill(mine, -1), -1)
    out.masked_fill_(~mine, -1)
    row, col = (mine & (out < 0)).nonzero(as_tuple=True)
    out[row, col] = free[: len(row)].to(torch.int32)
    s["refs_out"][free[: len(row)]] = 1
    s["table_out"].copy_(out)
    _copy_plain(s)


def _compact_plain(s):
    refs, dev = s["refs"], s["refs"].device
    used = refs > 0
    n = used.sum()
    at = torch.arange(len(refs), device=dev)
    frm = (used & (at >= n)).nonzero()[:, 0]
    to = (~used & (at < n)).nonzero()[:, 0]
    s["moves"][: len(frm)] = torch.stack((frm, to), -1).to(torch.int32)
    s["n_moves"].fill_(len(frm))
    s["n_used"].copy_(n)
    now = at.to(torch.int32)
    now[frm] = to.to(torch.int32)
    s["table_out"].copy_(torch.where(s["table"] >= 0, now[s["table"].clamp(min=0).long()], -1))
    s["refs_out"].copy_(refs)
    s["refs_out"][to] = refs[frm]
    s["refs_out"][frm] = 0
    _copy_plain(s)


def _turn_plain(x, gamma, s, row):
    """Norm, then the rotation by each pair's row of the tables, in 32 bits."""
    c = s["case"]
    D = x.shape[-1]
    x = x.float()
    if gamma is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gamma
    pair = torch.arange(D // 2, device=x.device)
    cos, sin = s["cos"][row, pair][:, :, None], s["sin"][row, pair][:, :, None]
    stays = s["axis_of"] == 3
    cos, sin = cos.masked_fill(stays, 1.0), sin.masked_fill(stays, 0.0)
    if c["rope"] == "interleaved":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    a, b = x.chunk(2, dim=-1)
    return torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)


def _axes_plain(s):
    c = s["case"]
    B, S = c["B"], c["S"]
    axis = torch.where(s["axis_of"] == 3, 0, s["axis_of"])
    row = s["positions"][:, :, axis].long()                               # [B, S, D/2]
    if c["into"] == "packed":
        s["q_out"].copy_(_turn_plain(s["q"], s["gq"], s, row))
        s["k_out"].copy_(_turn_plain(s["k"], s["gk"], s, row))
        return
    step = torch.arange(S, device=row.device)[None, :]
    n = torch.full_like(s["lens"], S) if s["new_lens"] is None else s["new_lens"]
    valid = step < n[:, None]
    at = torch.where(valid, s["lens"][:, None] + step, 0).long()
    page, slot = s["table"].gather(1, at // PAGE).long()[valid], (at % PAGE)[valid]
    k = _turn_plain(s["k"], s["gk"], s, row)[valid]                       # [tokens, Hkv, D]
    for cache, x, scale in ((s["kc"], k, s["ks"]), (s["vc"], s["v"].float()[valid], s["vs"])):
        if scale is not None:
            x = (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        _bytes_of(cache).permute(0, 2, 1, 3)[page, slot] = _bytes_of(x.to(cache.dtype))
    s["ksum"][page[slot == 0]] = 0.0
    s["ksum"].index_put_((page,), k, accumulate=True)
    s["q_out"][valid] = _turn_plain(s["q"], s["gq"], s, row)[valid].to(torch.bfloat16)
    s["lens_out"].copy_(s["lens"] + n)


# --------------------------------------------------------------------- run --

def _tree_own(sa, s):
    if "ws" not in s:                          # a program keeps its workspaces
        p = sa.make_cache_params(s["table"], q=s["q"], k_cache=s["kc"], v_cache=s["vc"])
        s["ws"] = torch.empty(sa.sa_attn_tree_workspace_bytes(p), dtype=torch.uint8,
                              device=s["q"].device)
    sa.sa_attn_tree(s["q"], s["kc"], s["vc"], s["table"], s["lens"], parents=s["parents"],
                    new_lens=s["new_lens"], row_ptr=s["row_ptr"], col_idx=s["col_idx"],
                    k_scale=s["ks"], v_scale=s["vs"], o=s["o"], lse=s["lse"], workspace=s["ws"])


def _accept_own(sa, s):
    sa.sa_cache_accept(s["kc"], s["vc"], s["table"], s["lens"], s["path"], s["path_lens"],
                       k_sum=s["ksum"], k_scale=s["ks"], lens_out=s["lens_out"])


def _fork_own(sa, s):
    if "ws" not in s:
        s["ws"] = torch.empty(sa.sa_pages_workspace_bytes(
            s["refs"].numel(), max(s["table"].shape[0], s["table_out"].shape[0])),
            dtype=torch.uint8, device=s["refs"].device)
    sa.sa_pages_fork(s["table"], s["lens"], s["refs"], s["src"], table_out=s["table_out"],
                     lens_out=s["lens_out"], refs_out=s["refs_out"], moves=s["moves"],
                     n_moves=s["n_moves"], workspace=s["ws"])
    sa.sa_pages_resize(s["table_out"], s["refs_out"], s["lens_out"], more=1, workspace=s["ws"])
    sa.sa_cache_copy(s["kc"], s["vc"], s["moves"], s["n_moves"], k_sum=s["ksum"])


def _compact_own(sa, s):
    if "ws" not in s:
        s["ws"] = torch.empty(sa.sa_pages_workspace_bytes(s["refs"].numel(), s["table"].shape[0]),
                              dtype=torch.uint8, device=s["refs"].device)
    sa.sa_pages_compact(s["table"], s["refs"], table_out=s["table_out"], refs_out=s["refs_out"],
                        moves=s["moves"], n_moves=s["n_moves"], n_used=s["n_used"],
                        workspace=s["ws"])
    sa.sa_cache_copy(s["kc"], s["vc"], s["moves"], s["n_moves"], k_sum=s["ksum"])


def _axes_own(sa, s):
    c = s["case"]
    if c["into"] == "packed":
        if "ws" not in s:
            s["ws"] = torch.empty(sa.sa_route_workspace_bytes(sa.make_params(s["q"], s["k"])),
                                  dtype=torch.uint8, device=s["q"].device)
        sa.sa_qk_prologue(s["q"], s["k"], s["gq"], s["gk"], 1e-6, s["cos"], s["sin"],
                          qk_norm=c["norm"], positions=s["positions"], axes=s["axes"],
                          q_out=s["q_out"], k_out=s["k_out"], workspace=s["ws"])
    else:
        sa.sa_cache_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens"], q=s["q"],
                           q_out=s["q_out"], new_lens=s["new_lens"], qk_norm=c["norm"],
                           gamma_q=s["gq"], gamma_k=s["gk"], eps=1e-6, cos=s["cos"], sin=s["sin"],
                           rope=c["rope"], positions=s["positions"], axes=s["axes"],
                           k_scale=s["ks"], v_scale=s["vs"], k_sum=s["ksum"],
                           lens_out=s["lens_out"])


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import block_sparse_attention_sa_gb300 as sa
        {"tree": _tree_own, "accept": _accept_own, "fork": _fork_own, "compact": _compact_own,
         "axes": _axes_own}[op](sa, s)
    else:
        {"tree": _tree_plain, "accept": _accept_plain, "fork": _fork_plain,
         "compact": _compact_plain, "axes": _axes_plain}[op](s)
    names = {"tree": ("o", "lse"), "accept": ("kc", "vc", "ksum", "lens_out"),
             "fork": ("table_out", "lens_out", "refs_out", "n_moves", "kc", "vc", "ksum"),
             "compact": ("table_out", "refs_out", "n_used", "n_moves", "kc", "vc", "ksum"),
             "axes": (("q_out", "k_out") if state["case"].get("into") == "packed" else
                      ("kc", "vc", "ksum", "q_out", "lens_out"))}
    return {name: s[name] for name in names[op]}


# -------------------------------------------------------------------- work --

def work(case):
    op, B, Hkv, D = case["op"], case["B"], case["Hkv"], case["D"]
    mean = case.get("past", 0) * (0.625 if case["ragged"] else 1.0)       # tokens of a sequence
    kv = 1 if case.get("fmt") == "fp8" else 2
    S = case.get("S", 1)
    tokens = B * S * (0.5 if S > 1 and case["ragged"] else 1.0)
    by = fl = 0.0
    if op == "tree":
        H = case["H"]
        keys = min(mean, PAGE * case["budget"]) if case["budget"] else mean
        by = B * (keys + S) * Hkv * D * 2 * kv + tokens * H * (4 * D + 4)
        fl = tokens * (keys + S / 2) * H * D * 4
    elif op == "accept":
        moved = 0.3 * tokens + B
        by = moved * Hkv * D * 4 * kv + B * Hkv * D * (4 + 32 * kv)
        fl = B * 32 * Hkv * D
    elif op == "fork":
        N = case["N"]
        pages = case["past"] / PAGE + 2
        share = [math.sqrt((b + 1) / B) - math.sqrt(b / B) for b in range(B)]
        copies = 15 / 16 * N - sum(1 - (1 - 15 / 16 * x) ** N for x in share)
        by = copies * (PAGE * 4 * kv + 8) * Hkv * D + 8 * N * pages + 8 * (B * pages + N)
        fl = N * pages
    elif op == "compact":
        used = B * mean / PAGE
        pages = B * case["past"] / PAGE / case["fill"]
        by = used * (1 - used / pages) * (PAGE * 4 * kv + 8) * Hkv * D + 8 * pages + 8 * used
        fl = pages
    else:
        H = case["H"]
        by = tokens * (H + Hkv) * D * 4 + tokens * 12
        if case["into"] == "cache":
            by = tokens * (H * D * 4 + Hkv * D * (4 + 2 * kv) + 12) + \
                max(B, tokens / PAGE) * Hkv * D * 8
        fl = tokens * (H + Hkv) * D * 8
    return {"bytes": by, "flops": fl}


# ------------------------------------------------------------------- exact --

def _exact_tree(s):
    """Token by token of the drafts: the set that each one sees."""
    c = s["case"]
    B, S, H, Hkv, D = c["B"], c["S"], c["H"], c["Hkv"], c["D"]
    G, dev = H // Hkv, s["q"].device
    o, lse = s["o"].double(), s["lse"].double()
    rp = None if s["row_ptr"] is None else s["row_ptr"].tolist()
    for b in range(B):
        base = int(s["lens"][b])
        n = S if s["new_lens"] is None else int(s["new_lens"][b])
        up = list(range(-1, S - 1)) if s["parents"] is None else s["parents"][b].tolist()
        sees = torch.zeros((n, n), dtype=torch.bool)
        for t in range(n):
            a = t
            while a >= 0:
                sees[t, a] = True
                a = up[a]
        sees = sees.to(dev)
        for g in range(Hkv):
            pages = torch.arange((base + n + PAGE - 1) // PAGE, device=dev)
            if rp is not None:
                listed_ = s["col_idx"][rp[b * Hkv + g]:rp[b * Hkv + g + 1]].long()
                pages = torch.cat((listed_, pages[base // PAGE:]))
            ids = s["table"][b][pages].long()
            tok = (pages[:, None] * PAGE + torch.arange(PAGE, device=dev)).flatten()
            tok = tok[tok < base + n]
            k, v = (_bytes_of(x)[ids, g].view(x.dtype).reshape(-1, D)[: len(tok)].double()
                    for x in (s["kc"], s["vc"]))
            if s["ks"] is not None:
                k, v = k * s["ks"][g].double(), v * s["vs"][g].double()
            q = s["q"][b, :n, g * G:(g + 1) * G].double()
            x = torch.matmul(q.reshape(-1, D), k.T).view(n, G, len(tok)) / math.sqrt(D)
            ok = (tok < base)[None, :].repeat(n, 1)
            ok[:, tok >= base] = sees[:, tok[tok >= base] - base]
            x = x.masked_fill(~ok[:, None, :], -math.inf)
            lse[b, g * G:(g + 1) * G, :n] = torch.logsumexp(x, -1).T
            o[b, :n, g * G:(g + 1) * G] = torch.softmax(x, -1) @ v
    return {"o": o, "lse": lse}


def _exact_accept(s):
    c = s["case"]
    kc, vc, ksum = s["kc"].double(), s["vc"].double(), s["ksum"].double()
    lens, table = s["lens"].tolist(), s["table"].tolist()
    end = s["lens"].clone()
    for b in range(c["B"]):
        for i, a in enumerate(s["path"][b, : int(s["path_lens"][b])].tolist()):
            f, t = lens[b] + a, lens[b] + i
            for x in (kc, vc):
                x[table[b][t // PAGE], :, t % PAGE] = x[table[b][f // PAGE], :, f % PAGE].clone()
        end[b] += s["path_lens"][b]
        for j in range(lens[b] // PAGE, -(-int(end[b]) // PAGE)):
            x = kc[table[b][j], :, : min(PAGE, int(end[b]) - j * PAGE)].sum(1)
            ksum[table[b][j]] = x if s["ks"] is None else x * s["ks"].double()[:, None]
    return {"kc": kc, "vc": vc, "ksum": ksum, "lens_out": end}


def _exact_axes(s):
    c = s["case"]
    D, axis = c["D"], s["axis_of"].tolist()

    def turned(x, gamma, pos):                 # [tokens, heads, D], [tokens, 3]
        x = x.double()
        if gamma is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * gamma.double()
        y = x.clone()
        for i in range(sum(s["axes"])):
            lo, hi = (2 * i, 2 * i + 1) if c["rope"] == "interleaved" else (i, i + D // 2)
            at = pos[:, axis[i]].long()
            co, si = s["cos"][at, i].double()[:, None], s["sin"][at, i].double()[:, None]
            y[..., lo] = x[..., lo] * co - x[..., hi] * si
            y[..., hi] = x[..., lo] * si + x[..., hi] * co
        return y

    if c["into"] == "packed":
        return {"q_out": torch.stack([turned(x, s["gq"], p) for x, p in zip(s["q"], s["positions"])]),
                "k_out": torch.stack([turned(x, s["gk"], p) for x, p in zip(s["k"], s["positions"])])}
    kc, vc, ksum, q_out = (s[n].double() for n in ("kc", "vc", "ksum", "q_out"))
    lens, table, end = s["lens"].tolist(), s["table"].tolist(), s["lens"].clone()
    for b in range(c["B"]):
        n = c["S"] if s["new_lens"] is None else int(s["new_lens"][b])
        end[b] += n
        pos = s["positions"][b, :n]
        q_out[b, :n] = turned(s["q"][b, :n], s["gq"], pos)
        k, v = turned(s["k"][b, :n], s["gk"], pos), s["v"][b, :n].double()
        t = 0
        while t < n:
            j, slot = divmod(lens[b] + t, PAGE)
            m, p = min(PAGE - slot, n - t), table[b][j]
            for cache, x, sc in ((kc, k, s["ks"]), (vc, v, s["vs"])):
                x = x[t:t + m].transpose(0, 1)
                if sc is not None:
                    x = (x / sc.double()[:, None, None]).clamp(-E4M3_MAX, E4M3_MAX)
                cache[p, :, slot:slot + m] = x
            ksum[p] = k[t:t + m].sum(0) + (ksum[p] if slot else 0)
            t += m
    return {"kc": kc, "vc": vc, "ksum": ksum, "q_out": q_out, "lens_out": end}


def _exact_fork(s):
    """Row by row, with lists."""
    c = s["case"]
    table, refs, lens = s["table"].tolist(), s["refs"].tolist(), s["lens"].tolist()
    free = [p for p, r in enumerate(refs) if r == 0]
    taken, rows, ends, moves = set(), [], [], []
    for b in s["src"].tolist():
        row, n = ([-1] * len(table[0]), 0) if b < 0 else (list(table[b]), lens[b])
        if b in taken and b >= 0:
            whole = n // PAGE
            row = row[:whole] + [-1] * (len(row) - whole)
            if n % PAGE:
                row[whole] = free.pop(0)
                moves.append((table[b][whole], row[whole]))
        taken.add(b)
        rows.append(row)
        ends.append(n)
    kc, vc, ksum = (s[n].double() for n in ("kc", "vc", "ksum"))
    for a, b in moves:
        for x in (kc, vc, ksum):
            x[b] = x[a]
    return {"table_out": None, "lens_out": torch.tensor(ends, dtype=torch.int32), "refs_out": None,
            "n_moves": torch.tensor([len(moves)], dtype=torch.int32), "kc": kc, "vc": vc,
            "ksum": ksum}


def _exact_compact(s):
    used = [p for p, r in enumerate(s["refs"].tolist()) if r]
    taken = set(used)
    holes = [p for p in range(len(used)) if p not in taken]
    late = [p for p in used if p >= len(used)]
    kc, vc, ksum = (s[n].double() for n in ("kc", "vc", "ksum"))
    to = dict(zip(late, holes))
    for a, b in to.items():
        for x in (kc, vc, ksum):
            x[b] = x[a]
    table = [[to.get(p, p) for p in row] for row in s["table"].tolist()]
    before = s["refs"].tolist()
    refs = before[: len(used)] + [0] * (len(before) - len(used))
    for a, b in to.items():
        refs[b] = before[a]
    return {"table_out": torch.tensor(table, dtype=torch.int32),
            "refs_out": torch.tensor(refs, dtype=torch.int32),
            "n_used": torch.tensor([len(used)], dtype=torch.int32),
            "n_moves": torch.tensor([len(late)], dtype=torch.int32), "kc": kc, "vc": vc, "ksum": ksum}


def exact(case, seed):
    """The operators' definitions in 64 bits."""
    s = prepare(case, seed)
    return {"tree": _exact_tree, "accept": _exact_accept, "fork": _exact_fork,
            "compact": _exact_compact, "axes": _exact_axes}[case["op"]](s)
